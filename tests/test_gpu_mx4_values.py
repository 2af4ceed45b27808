"""Every code under every scale byte, dequantised: what a stored pair stands for, rounded once to the output's type."""
import numpy as np
import pytest
import torch

import lowp_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu


def every_pair(fmt):
    """(matrix, its values in 64 bits): row r holds the 16 codes under scale byte r."""
    rows, K = (256, 32) if fmt == "mxfp4" else (128, 16)  # a sign bit in an E4M3 scale byte is never stored
    code = np.tile(np.arange(16, dtype=np.uint8), K // 16)
    codes = np.zeros((rows, 32), dtype=np.uint8)
    codes[:, : K // 2] = code[0::2] | code[1::2] << 4
    scales = np.zeros(ozk.mx4_scale_bytes(rows, K, fmt), dtype=np.uint8)
    r = np.arange(rows)
    scales[r // 128 * 512 + r % 32 * 16 + r // 32 % 4 * 4] = r
    q = ozk.Mx4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), rows, K, fmt)
    c = np.broadcast_to(code, (rows, K))
    return q, ref.values(c & 7, c >= 8, r[:, None].astype(np.uint8), fmt, K)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_every_pair_in_64_bits(fmt):
    q, want = every_pair(fmt)
    got = ozk.mx4_dequantize(q, torch.float64).cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isfinite(got[-2]).all()  # the largest scale


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_every_pair_rounded(fmt, dtype):
    """Values beyond a type's range become infinite, as its rounding has it."""
    q, want = every_pair(fmt)
    got = ozk.mx4_dequantize(q, dtype).double().cpu().numpy()
    rounded = torch.from_numpy(want).float().to(dtype).double().numpy()  # 64 to 32 bits is exact or infinite here
    assert np.array_equal(got, rounded, equal_nan=True)


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 1), (2, 0), (4, 4)])
def test_every_pair_at_any_alignment(offset, pad):
    q, want = every_pair("mxfp4")
    buf = torch.zeros(offset + 256 * (32 + pad), device="cuda", dtype=torch.float64)
    out = buf[offset:].view(256, 32 + pad)[:, :32]
    ozk.mx4_dequantize(q, out=out)
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("alpha", [float("inf"), float("nan"), -1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_of_no_terms_are_zero(alpha, dtype):
    """An empty sum is zero whatever alpha is: nothing is multiplied."""
    e, w = ozk.mx4_quantize(torch.empty(5, 0, device="cuda")), ozk.mx4_quantize(torch.empty(3, 7, 0, device="cuda"))
    out = ozk.mx4_gemm(e, e, alpha=alpha, out_dtype=dtype)
    assert torch.equal(out, torch.zeros(5, 5, device="cuda", dtype=dtype)) and not bool(out.signbit().any())
    x = ozk.mx4_quantize(torch.empty(5, 0, device="cuda"), offsets=torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda"))
    out = torch.full((5, 7), 9.0, device="cuda", dtype=dtype)
    ozk.mx4_grouped_gemm(x, w, alpha=alpha, out=out)
    assert torch.equal(out, torch.zeros_like(out))


def test_scales_at_ties_and_their_neighbours():
    """amax / 6 at and next to every boundary between two E4M3 scales, in fp32: one unit below a tie is below it, although a
    product with 1/6 would round onto the tie."""
    ties = (ref.E4M3[:-1] + ref.E4M3[1:]) / 2
    at = (6 * ties).astype(np.float32)  # exact
    assert np.array_equal(at.astype(np.float64), 6 * ties)
    tops = [at]
    for to in (np.float32(0), np.float32(np.inf)):
        v = at
        for _ in range(3):
            v = np.nextafter(v, to)
            tops.append(v)
    x = np.zeros((len(tops) * len(ties), 16), dtype=np.float32)
    x[:, 3] = np.concatenate(tops)
    x[:, 7] = -x[:, 3] / 3
    q = ozk.mx4_quantize(torch.from_numpy(x).cuda(), "nvfp4")
    code, neg, byte = ref.quantize(x, "nvfp4")
    assert np.array_equal(ref.stored_scales(q.scales.cpu().numpy(), len(x), 16, "nvfp4", [0, len(x)]), byte)
    want = ref.values(code, neg, byte, "nvfp4", 16)
    assert np.array_equal(ozk.mx4_dequantize(q, torch.float64).cpu().numpy(), want)
