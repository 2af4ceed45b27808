"""The backward pass of the gated product through its C entry point, into
buffers whose every byte is known before: what is written, what is cleared and
what is left alone; and the same bits every time."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu


def normal(*shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("starts", [[0, 9, 9, 49], [3, 12, 12, 52], [3, 3, 3, 3], [0, 0, 40, 58], [58, 58, 58, 58]])
@pytest.mark.parametrize("left,pad", [(0, 0), (1, 5), (8, 16), (3, 0)])
@pytest.mark.parametrize("H,K", [(61, 72), (64, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_in_no_group_are_cleared_and_nothing_else(starts, left, pad, H, K, dtype):
    """dX starts `left` elements into rows of left + K + pad: NaN before the call, zeros in rows of no group after it, its
    surroundings as they were; dpre untouched in those rows; dW whole, zeros for groups without rows."""
    T, groups = 58, 3
    x, w = normal(T, K, seed=1, dtype=dtype), normal(groups, 2 * H, K, seed=2, dtype=dtype)
    dh, slopes = normal(T, H, seed=3, dtype=dtype), normal(2, T, H, seed=4, dtype=torch.float32)
    offsets = torch.tensor(starts, dtype=torch.int32, device="cuda")
    nan = float("nan")
    ldp = -(-2 * H // 8) * 8
    dpre = torch.full((T, ldp), nan, dtype=dtype, device="cuda")
    room = torch.full((T, left + K + pad), nan, dtype=dtype, device="cuda")
    dx = room[:, left: left + K]
    wide = torch.full((groups, 2 * H, K + pad), nan, dtype=dtype, device="cuda")
    dw = wide[:, :, :K]
    torch.cuda.synchronize()
    rc = ozk.lib().ozk_grouped_gated_gemm_grad(
        T, H, K, groups, offsets.data_ptr(), dh.data_ptr(), H, slopes.data_ptr(), H, T * H, x.data_ptr(), K, w.data_ptr(), K,
        2 * H * K, {torch.bfloat16: ozk.OZK_BF16, torch.float16: ozk.OZK_F16}[dtype], dpre.data_ptr(), ldp, dx.data_ptr(),
        left + K + pad, dw.data_ptr(), K + pad, 2 * H * (K + pad), None)
    torch.cuda.synchronize()
    assert rc == 0
    inner, outer = slice(starts[0], starts[-1]), [slice(0, starts[0]), slice(starts[-1], T)]
    for rows in outer:
        assert not dx[rows].any() and bool((dx[rows] == 0).all())
        assert bool(torch.isnan(dpre[rows]).all())
    assert bool(torch.isnan(room[:, :left]).all()) and bool(torch.isnan(room[:, left + K:]).all())
    assert bool(torch.isnan(wide[:, :, K:]).all()) and bool(torch.isnan(dpre[:, 2 * H:]).all())
    want = torch.cat((dh.float() * slopes[0], dh.float() * slopes[1]), dim=1).to(dtype)
    assert torch.equal(dpre[inner, : 2 * H], want[inner])
    clean = torch.zeros(T, ldp, dtype=dtype, device="cuda")
    clean[:, : 2 * H] = want
    clean = clean[:, : 2 * H]
    assert torch.equal(dx[inner], ozk.grouped_gemm_dx(clean, w, offsets)[inner])
    assert torch.equal(dw, ozk.grouped_gemm_dw(clean, x, offsets))
    for e in range(groups):
        assert bool((dw[e] == 0).all()) == (starts[e] == starts[e + 1])
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("counts,H,K", [([130, 3, 0, 64], 136, 264), ([700, 0, 260], 296, 520), ([900, 1100], 1040, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_same_bits_every_time(counts, H, K, dtype):
    T = sum(counts)
    x, w = normal(T, K, seed=1, dtype=dtype).requires_grad_(), normal(len(counts), 2 * H, K, seed=2, dtype=dtype).requires_grad_()
    dh = normal(T, H, seed=3, dtype=dtype)
    starts = [sum(counts[:i]) for i in range(len(counts) + 1)]
    offsets = torch.tensor(starts, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(4):
        h = ozk.grouped_gated_gemm(x, w, offsets)
        got = (h.detach(), *torch.autograd.grad(h, (x, w), dh))
        first = first or got
        for a, b in zip(first, got):
            assert torch.equal(a, b)
