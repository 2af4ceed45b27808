"""Products of rows grouped by expert and their gradients on the GPU, against
64-bit products group by group.

A result sums K terms (the gradient of w: a group's rows) in fp32; every one
of its at most K additions is off by at most 2^-23 of the magnitudes summed so
far, so it lies within K 2^-23 sum |a b| of the exact one, plus its own
rounding.  With small whole numbers every sum is exact and results are equal."""
import numpy as np
import pytest
import torch

import lowp_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SHAPES = [([1], 8, 8), ([5, 0, 17], 128, 64), ([130, 3, 0, 64], 264, 136), ([300, 1], 72, 1032), ([1] * 24, 512, 256),
          ([16, 15, 0, 0, 49, 128, 129], 136, 392), ([700, 0, 260], 520, 584), ([61] * 30, 520, 520)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(*shape, seed, dtype):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


def whole(*shape, seed, dtype):
    return torch.randint(-2, 3, shape, generator=gen(seed), device="cuda").to(dtype)


def starts_of(counts):
    return np.cumsum([0] + counts).tolist()


def device_offsets(starts):
    return torch.tensor(starts, dtype=torch.int32, device="cuda")


def near(got, exact, mags, terms, dtype):
    got = got.double().cpu().numpy()
    assert got.shape == exact.shape
    bound = terms * 2.0 ** -23 * mags + ROUND[dtype] * np.abs(exact) + 2.0 ** -24
    assert np.all(np.abs(got - exact) <= bound)


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("wide", [False, True])
def test_products_and_gradients(counts, N, K, dtype, wide):
    starts, G = starts_of(counts), len(counts)
    T, off = starts[-1], device_offsets(starts_of(counts))
    out = torch.float32 if wide else dtype
    x, dy = normal(T, K, seed=1, dtype=dtype), normal(T, N, seed=2, dtype=dtype)
    w = (normal(G, N, K, seed=3, dtype=torch.float32) / 16).to(dtype)
    hx, hdy, hw = (t.double().cpu().numpy() for t in (x, dy, w))
    near(ozk.grouped_gemm(x, w, off, out_dtype=out), ref.grouped(hx, hw, starts),
         ref.grouped(np.abs(hx), np.abs(hw), starts), K, out)
    near(ozk.grouped_gemm_dx(dy, w, off, out_dtype=out), ref.grouped_dx(hdy, hw, starts),
         ref.grouped_dx(np.abs(hdy), np.abs(hw), starts), N, out)
    near(ozk.grouped_gemm_dw(dy, x, off, out_dtype=out), ref.grouped_dw(hdy, hx, starts),
         ref.grouped_dw(np.abs(hdy), np.abs(hx), starts), max(counts), out)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("counts,N,K", [([900, 1300, 0, 77], 1544, 1160), ([300] * 12, 776, 1032)])
def test_many_tiles_per_cta_exact(counts, N, K):
    """Several waves of tiles on both tile forms, whole numbers: every output equal, and the same in 16 bits."""
    starts, G = starts_of(counts), len(counts)
    T, off, dtype = starts[-1], device_offsets(starts_of(counts)), torch.bfloat16
    x, dy, w = whole(T, K, seed=1, dtype=dtype), whole(T, N, seed=2, dtype=dtype), whole(G, N, K, seed=3, dtype=dtype)
    for got, want in ((lambda t: ozk.grouped_gemm(x, w, off, out_dtype=t),
                       torch.cat([x[a:b].double() @ w[g].double().t() for g, (a, b) in enumerate(zip(starts, starts[1:]))])),
                      (lambda t: ozk.grouped_gemm_dx(dy, w, off, out_dtype=t),
                       torch.cat([dy[a:b].double() @ w[g].double() for g, (a, b) in enumerate(zip(starts, starts[1:]))])),
                      (lambda t: ozk.grouped_gemm_dw(dy, x, off, out_dtype=t),
                       torch.stack([dy[a:b].double().t() @ x[a:b].double() for a, b in zip(starts, starts[1:])]))):
        assert torch.equal(got(torch.float32).double(), want)
        assert torch.equal(got(dtype), want.to(dtype))


def test_gradients_against_differences():
    """y is linear: <r, y(x + d) - y(x)> = <dx(r), d> and <r, y(w + e) - y(w)> = <dw(r), e>, exactly for whole numbers."""
    counts, N, K = [33, 0, 70, 5], 136, 72
    starts, G, dtype, wide = starts_of(counts), 4, torch.bfloat16, torch.float32
    T, off = starts[-1], device_offsets(starts_of(counts))
    x, d, r = whole(T, K, seed=1, dtype=dtype), whole(T, K, seed=2, dtype=dtype), whole(T, N, seed=3, dtype=dtype)
    w, e = whole(G, N, K, seed=4, dtype=dtype), whole(G, N, K, seed=5, dtype=dtype)
    y = lambda x, w: ozk.grouped_gemm(x, w, off, out_dtype=wide).double()  # noqa: E731
    dx, dw = ozk.grouped_gemm_dx(r, w, off, out_dtype=wide), ozk.grouped_gemm_dw(r, x, off, out_dtype=wide)
    assert float((r.double() * (y(x + d, w) - y(x, w))).sum()) == float((dx.double() * d.double()).sum())
    assert float((r.double() * (y(x, w + e) - y(x, w))).sum()) == float((dw.double() * e.double()).sum())


@pytest.mark.parametrize("counts", [[3, 0, 20, 1], [40, 90]])
def test_rows_outside_every_group(counts):
    """Rows before the first and after the last group: no result, no part in any sum, whatever they hold."""
    starts = (np.cumsum([0] + counts) + 7).tolist()
    G, T, N, K = len(counts), starts[-1] + 21, 136, 264
    off = device_offsets(starts)
    x, dy = whole(T, K, seed=1, dtype=torch.bfloat16), whole(T, N, seed=2, dtype=torch.bfloat16)
    w = whole(G, N, K, seed=3, dtype=torch.bfloat16)
    for t in (x, dy):
        t[:7], t[starts[-1]:] = float("nan"), float("inf")
    inside = slice(7, starts[-1])
    near_starts = [s - 7 for s in starts]
    hx, hdy, hw = (t.double().cpu().numpy() for t in (x[inside], dy[inside], w))
    y = torch.full((T, N), 9.0, device="cuda")
    ozk.grouped_gemm(x, w, off, out=y)
    assert np.array_equal(y[inside].cpu().numpy(), ref.grouped(hx, hw, near_starts))
    dx = torch.full((T, K), 9.0, device="cuda")
    ozk.grouped_gemm_dx(dy, w, off, out=dx)
    assert np.array_equal(dx[inside].cpu().numpy(), ref.grouped_dx(hdy, hw, near_starts))
    for t in (y, dx):
        assert bool((t[:7] == 9).all()) and bool((t[starts[-1]:] == 9).all())
    assert np.array_equal(ozk.grouped_gemm_dw(dy, x, off, out_dtype=torch.float32).cpu().numpy(),
                          ref.grouped_dw(hdy, hx, near_starts))


def test_nan_stays_in_its_group():
    """An Inf or NaN in one group's rows or weights reaches no other group, and in the products only its own row."""
    counts, N, K = [19, 45, 3, 64], 200, 136
    starts, G = starts_of(counts), 4
    T, off = starts[-1], device_offsets(starts_of(counts))
    x, dy = whole(T, K, seed=1, dtype=torch.bfloat16), whole(T, N, seed=2, dtype=torch.bfloat16)
    w = whole(G, N, K, seed=3, dtype=torch.bfloat16)
    y0, dx0, dw0 = ozk.grouped_gemm(x, w, off), ozk.grouped_gemm_dx(dy, w, off), ozk.grouped_gemm_dw(dy, x, off)
    x[20], dy[63] = float("nan"), float("inf")  # first and last row of group 1
    y, dx, dw = ozk.grouped_gemm(x, w, off), ozk.grouped_gemm_dx(dy, w, off), ozk.grouped_gemm_dw(dy, x, off)
    rows = torch.arange(T, device="cuda")
    assert torch.equal(y[rows != 20], y0[rows != 20]) and bool(y[20].isnan().all())
    assert torch.equal(dx[rows != 63], dx0[rows != 63]) and not bool(torch.isfinite(dx[63]).any())
    for g in (0, 2, 3):
        assert torch.equal(dw[g], dw0[g])
    w[2, 7, 9] = float("nan")
    x[20] = 0
    y = ozk.grouped_gemm(x, w, off)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[64:67, 7] = True
    assert torch.equal(y.isnan(), bad)


@pytest.mark.parametrize("pad", [8, 40])
def test_strides(pad):
    """Leading dimensions and group strides wider than the matrices, inputs and outputs."""
    counts, N, K = [70, 0, 9], 104, 88
    starts, G = starts_of(counts), 3
    T, off = starts[-1], device_offsets(starts_of(counts))

    def wide(*shape, seed):
        buf = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), device="cuda", dtype=torch.float16)
        view = buf[..., : shape[-1]]
        view.copy_(whole(*shape, seed=seed, dtype=torch.float16))
        return view

    x, dy, w = wide(T, K, seed=1), wide(T, N, seed=2), wide(2 * G, N, K, seed=3)[::2]
    hx, hdy, hw = (t.double().cpu().numpy() for t in (x, dy, w))
    for call, want, shape in ((lambda o: ozk.grouped_gemm(x, w, off, out=o), ref.grouped(hx, hw, starts), (T, N)),
                              (lambda o: ozk.grouped_gemm_dx(dy, w, off, out=o), ref.grouped_dx(hdy, hw, starts), (T, K)),
                              (lambda o: ozk.grouped_gemm_dw(dy, x, off, out=o), ref.grouped_dw(hdy, hx, starts), (G, N, K))):
        for extra in (0, 1, 8):
            buf = torch.full((*shape[:-1], shape[-1] + extra), 99.0, device="cuda", dtype=torch.float16)
            call(buf[..., : shape[-1]])
            assert np.array_equal(buf[..., : shape[-1]].cpu().numpy(), want.astype(np.float16))
            assert bool((buf[..., shape[-1]:] == 99).all())


def test_empty_sizes():
    off = device_offsets([0, 0, 0])
    e = lambda *s: torch.empty(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    assert ozk.grouped_gemm(e(0, 64), e(2, 32, 64), off).shape == (0, 32)
    assert ozk.grouped_gemm_dx(e(0, 32), e(2, 32, 64), off).shape == (0, 64)
    dw = torch.full((2, 32, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    ozk.grouped_gemm_dw(e(0, 32), e(0, 64), off, out=dw)
    assert bool((dw == 0).all())
    y = torch.full((3, 32), 5.0, device="cuda", dtype=torch.bfloat16)
    ozk.grouped_gemm(e(3, 0), e(2, 32, 0), device_offsets([0, 1, 3]), out=y)
    assert bool((y == 0).all())


@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [-5, 10, 20, 60], [0, 10, 20, 1000], [60, 0, 60, 0]])
def test_bad_offsets_are_reported(bad):
    """Offsets out of range or running backwards: cut, never followed; reported, and cleared by the report."""
    T, N, K, G = 60, 64, 64, 3
    x, w = whole(T, K, seed=1, dtype=torch.bfloat16), whole(G, N, K, seed=2, dtype=torch.bfloat16)
    ozk.grouped_gemm(x, w, device_offsets(bad))
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    assert ozk.ozk_stream_status() == 0
    ozk.grouped_gemm_dw(x, x, device_offsets(bad))
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, offsets=device_offsets(bad)), ozk.mx4_quantize(w))
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    want = ref.grouped(x.double().cpu().numpy(), w.double().cpu().numpy(), [0, 1, 30, 60])
    got = ozk.grouped_gemm(x, w, device_offsets([0, 1, 30, 60]), out_dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy(), want) and ozk.ozk_stream_status() == 0


def test_bad_offsets_that_name_rows_many_times():
    """Every second group all rows again: only the first keeps them, and there are no more tiles than rows allow."""
    T, N, K, G = 500, 136, 72, 600
    x, w = whole(T, K, seed=1, dtype=torch.bfloat16), whole(G, N, K, seed=2, dtype=torch.bfloat16)
    off = device_offsets([0, T] * (G // 2) + [0])
    y = ozk.grouped_gemm(x, w, off, out_dtype=torch.float32)
    dw = ozk.grouped_gemm_dw(y.to(torch.bfloat16), x, off, out_dtype=torch.float32)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    assert torch.equal(y.double(), x.double() @ w[0].double().t())
    assert bool((dw[1:] == 0).all()) and bool((dw[0] != 0).any())


def test_most_groups():
    G, N, K = ozk.OZK_MAX_GROUPS, 32, 64
    counts = [(g * 7) % 5 for g in range(G)]
    starts = starts_of(counts)
    x, w = whole(starts[-1], K, seed=1, dtype=torch.bfloat16), whole(G, N, K, seed=2, dtype=torch.bfloat16)
    got = ozk.grouped_gemm(x, w, device_offsets(starts), out_dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy(), ref.grouped(x.double().cpu().numpy(), w.double().cpu().numpy(), starts))
    dw = ozk.grouped_gemm_dw(got.to(torch.bfloat16) * 0 + 1, x, device_offsets(starts), out_dtype=torch.float32)
    want = torch.stack([x[a:b].float().sum(dim=0) for a, b in zip(starts, starts[1:])])
    assert torch.equal(dw, want[:, None, :].expand(G, N, K))


def test_sizes_past_32_bits():
    """Rows and results of more than 2^31 elements, and weights whose last group lies past 2^31 elements."""
    T, N, K = 300_000, 7200, 64
    x = whole(1000, K, seed=1, dtype=torch.bfloat16).repeat(300, 1)
    w = whole(1, N, K, seed=2, dtype=torch.bfloat16).repeat(2, 1, 1)
    off = device_offsets([0, 1000, T])
    y = ozk.grouped_gemm(x, w, off)
    assert torch.equal(y[-1000:], y[:1000])
    dx = ozk.grouped_gemm_dx(y, w, off, out_dtype=torch.float32)
    assert torch.equal(dx[-1000:], dx[:1000])
    dw = ozk.grouped_gemm_dw(y, x, device_offsets([0, T - 1000, T]), out_dtype=torch.float32)
    assert torch.equal(dw[1], ozk.grouped_gemm_dw(y[:1000], x[:1000], device_offsets([0, 1000]), out_dtype=torch.float32)[0])
    del y, dx, dw
    G, N, K = 20, 16384, 8192
    w = whole(1, N, K, seed=2, dtype=torch.bfloat16).expand(G, N, K).contiguous()
    x = whole(1, K, seed=1, dtype=torch.bfloat16).repeat(G, 1)
    y = ozk.grouped_gemm(x, w, device_offsets(list(range(G + 1))), out_dtype=torch.float32)
    assert torch.equal(y[-1], y[0]) and torch.equal(y[0].double(), w[0].double() @ x[0].double())


def test_other_streams_and_graphs():
    G, N, K, T = 4, 136, 264, 50
    x, w = whole(T, K, seed=1, dtype=torch.bfloat16), whole(G, N, K, seed=2, dtype=torch.bfloat16)
    off = device_offsets([0, 5, 5, 31, 50])
    want = ozk.grouped_gemm(x, w, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ozk.grouped_gemm(x, w, off, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ozk.grouped_gemm(x, w, off)
        dx = ozk.grouped_gemm_dx(y, w, off, out_dtype=torch.float32)
        dw = ozk.grouped_gemm_dw(y, x, off, out_dtype=torch.float32)
    off.copy_(torch.tensor([0, 20, 21, 21, 50], dtype=torch.int32))
    graph.replay()
    assert torch.equal(y, ozk.grouped_gemm(x, w, off))
    assert torch.equal(dx, ozk.grouped_gemm_dx(y, w, off, out_dtype=torch.float32))
    assert torch.equal(dw, ozk.grouped_gemm_dw(y, x, off, out_dtype=torch.float32))


def test_wrapper_refusals():
    x, w = torch.ones(8, 64, device="cuda", dtype=torch.bfloat16), torch.ones(2, 32, 64, device="cuda", dtype=torch.bfloat16)
    off = device_offsets([0, 4, 8])
    with pytest.raises(TypeError):
        ozk.grouped_gemm(x, w.half(), off)
    with pytest.raises(ozk.OzkError):
        ozk.grouped_gemm(x.float(), w.float(), off)
    with pytest.raises(ValueError):
        ozk.grouped_gemm(x[:, :32], w, off)
    with pytest.raises(ValueError):
        ozk.grouped_gemm(x, w, device_offsets([0, 8]))
    with pytest.raises(TypeError):
        ozk.grouped_gemm(x, w, off.long())
    with pytest.raises(ValueError):
        ozk.grouped_gemm(x, w.transpose(1, 2), off)
    with pytest.raises(ValueError):  # one row for all: nothing there to read at a row's distance
        ozk.grouped_gemm(x[:1].expand(8, 64), w, off)
    with pytest.raises(ValueError):  # as a sum's gradient comes
        ozk.grouped_gemm_dx(torch.ones(1, 1, device="cuda", dtype=torch.bfloat16).expand(8, 32), w, off)
    with pytest.raises(ValueError):
        ozk.grouped_gemm(x, w[:1].expand(2, 32, 64), off)
    with pytest.raises(ValueError):
        ozk.grouped_gemm(x, w, off.cpu())
    with pytest.raises(ozk.OzkError):
        ozk.grouped_gemm(x, w, off, out_dtype=torch.float16)
    with pytest.raises(ozk.OzkError) as e:  # rows of 60 elements: not 16-byte aligned
        ozk.grouped_gemm(torch.ones(8, 60, device="cuda", dtype=torch.bfloat16),
                         torch.ones(2, 32, 60, device="cuda", dtype=torch.bfloat16), off)
    assert e.value.status == ozk.OZK_ERR_UNSUPPORTED
    with pytest.raises(ozk.OzkError) as e:
        ozk.grouped_gemm(x, torch.ones(2, 64, 64, device="cuda", dtype=torch.bfloat16), off, out=x)
    assert e.value.status == ozk.OZK_ERR_INVALID_ARG
