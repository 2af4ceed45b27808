"""The bounded waits of the low-precision products, run out without a fault:
one stage's copies of a CTA's first tile are never issued (on a CTA pair: one
CTA's half of them) and the waits have a short limit.  The kernel has to latch
OZK_ERR_TIMEOUT, stop the CTA and its peer, wait for the copies in flight and
return; the other tiles are right, and so are the next calls, which could not
run if the aborted CTAs had kept their TMEM."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import build as ozk_build
from fp64_gemm_emulation_exponent_gb300 import ozk

COUNTS, N, K = [1000, 0, 130], 520, 1000  # dW: 16 stages a tile of group 0, the last with rows to clear


def whole(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.bfloat16)


def calls():
    """name -> (call with an output, its shape, tile rows of group 0 or None for all, columns, k-blocks of the first tile)"""
    starts = [0, 1000, 1000, 1130]
    T, off = starts[-1], torch.tensor(starts, dtype=torch.int32, device="cuda")
    x, dy, w = whole(T, K, seed=1), whole(T, N, seed=2), whole(3, N, K, seed=3)
    found = {
        "forward": (lambda out: ozk.grouped_gemm(x, w, off, out=out), (T, N), 16),
        "dx": (lambda out: ozk.grouped_gemm_dx(dy, w, off, out=out), (T, K), 9),
        "dw": (lambda out: ozk.grouped_gemm_dw(dy, x, off, out=out), (3, N, K), 16),
    }
    wide = 2600
    for fmt in ("nvfp4", "mxfp4"):
        a, b = ozk.mx4_quantize(whole(700, wide, seed=4), fmt), ozk.mx4_quantize(whole(N, wide, seed=5), fmt)
        found[fmt] = (lambda out, a=a, b=b: ozk.mx4_gemm(a, b, out=out), (700, N), 11)
    return found


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", ["first", "inside", "last"])
@pytest.mark.parametrize("pairs,cta", [(0, 0), (1, 0), (1, 1)])
@pytest.mark.parametrize("name", ["forward", "dx", "dw", "nvfp4", "mxfp4"])
def test_withheld_copies_run_a_wait_out_and_the_next_calls_are_right(name, pairs, cta, block, dtype):
    call, shape, blocks = calls()[name]
    want = torch.zeros(shape, device="cuda", dtype=dtype)
    call(want)
    assert ozk.ozk_stream_status() == 0
    out = torch.full(shape, float("nan"), device="cuda", dtype=dtype)
    ozk.ozk_withhold_next_product(pairs, cta, {"first": 0, "inside": 7, "last": blocks - 1}[block], 5000)
    call(out)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_TIMEOUT
    assert ozk.ozk_stream_status() == 0  # reading the status clears it
    # all but the first tile, which starts at the first row and column
    missing = out.isnan()
    flat = missing.view(-1, shape[-1])
    rows, cols = int(flat[:, 0].sum()), int(flat[0].sum())
    assert 0 < rows <= (256 if pairs else 128) and cols == (256 if pairs else 128)
    assert bool(flat[:rows, :cols].all()) and int(flat.sum()) == rows * cols
    assert torch.equal(out[~missing], want[~missing])
    for _ in range(2):
        out.fill_(float("nan"))
        call(out)
        assert ozk.ozk_stream_status() == 0
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("name", ["forward", "dx", "dw", "nvfp4", "mxfp4"])
def test_a_limit_alone_changes_nothing(name, pairs):
    call, shape, blocks = calls()[name]
    want, out = (torch.zeros(shape, device="cuda") for _ in range(2))
    call(want)
    for kblock in (-1, blocks):
        ozk.ozk_withhold_next_product(pairs, 0, kblock, 100000)
        call(out.fill_(7.0))
        assert ozk.ozk_stream_status() == 0
        assert torch.equal(out, want)


@pytest.fixture(scope="module")
def library():
    ozk_build.build()
    return ozk.lib()


def test_request_refusals(library):
    for bad in ((-1, 0, 0, 1000), (2, 0, 0, 1000), (0, 1, 0, 1000), (1, 2, 0, 1000), (0, -1, 0, 1000), (0, 0, -2, 1000),
                (0, 0, 0, 1000001)):
        assert library.ozk_withhold_next_product(*bad) == ozk.OZK_ERR_INVALID_ARG
    assert library.ozk_withhold_next_product(1, 1, 3, 1000) == ozk.OZK_OK
    assert library.ozk_withhold_next_product(0, 0, 0, 0) == ozk.OZK_OK  # taken back


@pytest.mark.gpu
def test_waits_for_a_tail_behind_many_tiles():
    """The warp that clears a group's last rows is ahead by all tiles without such rows: here by about 0.9 ms of them, where
    a tile takes under 0.1 ms.  A limit of 0.3 ms must not run out."""
    starts = [0, 16384, 16397]
    off = torch.tensor(starts, dtype=torch.int32, device="cuda")
    dy, x = whole(starts[-1], 8192, seed=1), whole(starts[-1], 8192, seed=2)
    want = ozk.grouped_gemm_dw(dy, x, off)
    ozk.ozk_withhold_next_product(1, 0, -1, 300)
    got = ozk.grouped_gemm_dw(dy, x, off)
    assert ozk.ozk_stream_status() == 0
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_waits_do_not_count_the_kernel_before():
    """A product without offsets may start while the kernel before it still runs (here 10 ms, on one SM): its limit of 2 ms
    is for its own work."""
    rows = 1 << 22
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    dy, x = whole(rows, 128, seed=1), whole(rows, 128, seed=2)
    a, b = ozk.mx4_quantize(whole(300, 640, seed=3)), ozk.mx4_quantize(whole(300, 640, seed=4))
    want = ozk.mx4_gemm(a, b)
    ozk.grouped_gemm_dw(dy, x, off)
    assert ozk.ozk_stream_status() == 0
    for pairs in (0, 1):
        ozk.grouped_gemm_dw(dy, x, off)
        ozk.ozk_withhold_next_product(pairs, 0, -1, 2000)
        got = ozk.mx4_gemm(a, b)
        assert ozk.ozk_stream_status() == 0
        assert torch.equal(got, want)
