"""Group offsets that lie outside the rows or run backwards, in every call of
the 4-bit matrices that takes them: reported by the call alone, and cut by one
rule (each start at least the end before it, all within the rows), so that
codes, scales and products agree on which group a row belongs to."""
import numpy as np
import pytest
import torch

import lowp_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
T, K, N = 300, 192, 136
BAD = [[0, 250, 20, 300], [-5, 10, 20, 300], [0, 10, 20, 1000], [300, 0, 300, 0], [7, 140, 130, 290], [0, 400, 10, 300],
       [-9, -3, -1, 200], [2 ** 31 - 1, -2 ** 31, 5, 130]]


def cut(offsets):
    out, at = [], 0
    for o in offsets:
        at = min(max(o, at), T)
        out.append(at)
    return out


def device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def whole(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("bad", BAD)
def test_each_call_reports_bad_offsets(fmt, bad):
    x = whole(T, K, seed=1)
    q = ozk.mx4_quantize(x, fmt, offsets=device(bad))
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    assert ozk.ozk_stream_status() == 0
    ozk.mx4_dequantize(q)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    good = ozk.mx4_quantize(x, fmt, offsets=device(cut(bad)))
    ozk.mx4_dequantize(good)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("bad", BAD)
def test_bad_offsets_are_cut_by_one_rule(fmt, bad):
    starts = cut(bad)
    x, w = whole(T, K, seed=1), ozk.mx4_quantize(whole(3, N, K, seed=2), fmt)
    q = ozk.mx4_quantize(x, fmt, offsets=device(bad))
    inside = np.arange(starts[0], starts[-1])
    code, neg, byte = ref.quantize(x.double().cpu().numpy(), fmt)
    assert np.array_equal(ref.stored_codes(q.codes.cpu().numpy(), K)[0][inside], code[inside])
    assert np.array_equal(ref.stored_scales(q.scales.cpu().numpy(), T, K, fmt, starts)[inside], byte[inside])
    rows = torch.full((T, K), 9.0, device="cuda")
    ozk.mx4_dequantize(q, out=rows)
    want = torch.full((T, K), 9.0, device="cuda")
    want[starts[0]: starts[-1]] = torch.from_numpy(ref.values(code, neg, byte, fmt, K)[inside]).float().cuda()
    assert torch.equal(rows, want)
    y = torch.full((T, N), 9.0, device="cuda")
    ozk.mx4_grouped_gemm(q, w, out=y)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    want = torch.full((T, N), 9.0, device="cuda")
    ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, fmt, offsets=device(starts)), w, out=want)
    assert torch.equal(y, want)
    assert ozk.ozk_stream_status() == 0


def test_most_groups():
    """As many offsets as there may be, the last one bad: found by blocks that have nothing else to do with it."""
    G = ozk.OZK_MAX_GROUPS
    starts = [min(g, T) for g in range(G)] + [T - 1]
    ozk.mx4_quantize(whole(T, K, seed=1), offsets=device(starts))
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    starts[-1] = T
    ozk.mx4_quantize(whole(T, K, seed=1), offsets=device(starts))
    assert ozk.ozk_stream_status() == 0
