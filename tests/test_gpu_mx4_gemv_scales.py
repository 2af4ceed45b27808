"""Products of a few rows with MXFP4 weights whose scale bytes are near the ends
of their range, and long sums.

Beside the K 2^-23 sum |x w| of the sums' roundings: a bf16 row is multiplied
by a power of two that brings the largest element of a chunk to 2^9 at least (or
by 2^127, if that is less), and a block's sum times its scale is rounded to a
multiple of 2^-149, twice with the sum so far: that is 2^-158 of the row's
largest element for each block of 32.  Each of up to 16 warps then takes its
sum's power of two back by two factors, and the second rounds to a multiple of
2^-149: 2^-150 (the first one's rounding, 2^-150 times the second factor, is below
2^-160 where that factor shrinks, and none where it grows); sums of such multiples
are exact.  16 (2^-150 + 2^-160) is below 2^-146 + 2^-150."""
import numpy as np
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def stored(rows, K, lo, hi, seed, codes=None):
    """An MXFP4 matrix of random codes under scale bytes lo to hi, and its values in 64 bits."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, K)) if codes is None else np.full((rows, K), codes)
    byte = rng.integers(lo, hi + 1, (rows, K // 32))
    packed = (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)
    tiles = K // 128
    scales = np.zeros((rows // 128 + 1, tiles, 32, 4, 4), np.uint8)
    r = np.arange(rows)
    scales[r // 128, :, r % 32, r // 32 % 4] = byte.reshape(rows, tiles, 4)
    q = ozk.Mx4(torch.from_numpy(packed).cuda(), torch.from_numpy(scales.reshape(-1)).cuda(), rows, K, "mxfp4")
    value = np.where(code >= 8, -GRID[code % 8], GRID[code % 8])
    return q, value * np.repeat(np.ldexp(1.0, byte - 127), 32, axis=1)


@pytest.mark.parametrize("T", [1, 5, 12])
@pytest.mark.parametrize("bytes_", [(0, 0), (0, 6), (1, 60)])
@pytest.mark.parametrize("power", [0, 100, -30])
def test_small_scales(T, bytes_, power):
    N, K = 70, 4096
    q, w = stored(N, K, *bytes_, seed=1)
    x = (torch.randn(T, K, generator=torch.Generator().manual_seed(2)) * 2.0 ** power).bfloat16()
    got = ozk.mx4_gemv(x.cuda(), q, out_dtype=torch.float32).double().cpu().numpy()
    X = x.double().numpy()
    want, mags = X @ w.T, np.abs(X) @ np.abs(w).T
    top = np.abs(X).max(axis=1, keepdims=True)
    bound = (K + 64) * 2.0 ** -23 * mags + K / 32 * 2.0 ** -158 * top
    bound += 2.0 ** -24 * (np.abs(want) + bound) + 2.0 ** -146 + 2.0 ** -149
    assert np.all(np.abs(got - want) <= bound)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("T", [2, 8, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,power", [(1 << 12, 97), (1 << 15, 94), (1 << 18, 91)])
def test_large_scales_and_long_sums(T, dtype, K, power):
    """The largest codes, one sign, rows that use all of the room above their scale: finite while 6 * 2^16 * 2^power * K is
    below 2^128."""
    assert 6 * 2.0 ** 16 * 2.0 ** power * K < 2.0 ** 128
    N = 40
    q, w = stored(N, K, power + 127, power + 127, seed=3, codes=7)
    x = torch.full((T, K), 127.5 if dtype == torch.bfloat16 else 65504.0)
    if dtype == torch.bfloat16:
        x[:, : K // 16] = 1.0  # the scale is made for these; the rest is 2^6 larger
    x = x.to(dtype).cuda()
    got = ozk.mx4_gemv(x, q, alpha=2.0 ** -30, out_dtype=torch.float32).double().cpu().numpy()
    want = 2.0 ** -30 * (x.double().cpu().numpy() @ w.T)
    assert np.all(np.abs(got - want) <= (K + 64) * 2.0 ** -23 * want + 2.0 ** -23 * want)
    assert ozk.ozk_stream_status() == 0
