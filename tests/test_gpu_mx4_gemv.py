"""Products of a few 16-bit rows with 4-bit weights on the GPU, plain and
gated, against 64-bit products of the stored values.

Operands and their products are exact, K terms are summed in fp32: a sum lies
within K 2^-23 sum |x w| of the exact one (each addition off by at most 2^-23
of the magnitudes summed so far; the additions that join the warps' and
panels' sums are among the K where K > 64 and counted as 64 more otherwise),
plus the result's own rounding.  The gated product's activation is off by up to 40
units of fp32 for |z| up to 14 (its argument rounded twice, the exponential off by
2 + 1.2 |z| units) and hands g's error on by at most 1.13 (the largest
derivative of the three)."""
import math

import numpy as np
import pytest
import torch

import lowp_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SIZES = [(1, 1, 1), (1, 16, 64), (2, 17, 100), (5, 1537, 2090), (8, 40, 4097), (9, 300, 1000), (16, 136, 640), (17, 70, 4500),
         (31, 9, 130), (40, 33, 260), (1, 5000, 129), (3, 20000, 64), (12, 8200, 200), (33, 8200, 72),
         (6, 4096, 320), (1, 4096, 256), (11, 4096, 192), (2, 1024, 96), (20, 2048, 128)]
_erf = np.vectorize(math.erf)


def normal(*shape, seed, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def act64(g, act):
    if act == "gelu":
        return g * 0.5 * (1 + _erf(g * math.sqrt(0.5)))
    z = g if act == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    return g / (1 + np.exp(-z))


def weights(rows, K, fmt, groups, seed):
    shape = (rows, K) if groups == 1 else (groups, rows, K)
    q = ozk.mx4_quantize(normal(*shape, seed=seed), fmt)
    return q, ozk.mx4_dequantize(q, torch.float64).cpu().numpy().reshape(groups, rows, K)


def near(got, exact, mags, K, dtype, gate=None):
    """gate: (act(g), g's magnitudes, u, u's magnitudes) of the gated product."""
    terms = (K + 64) * 2.0 ** -23
    if gate is None:
        bound = terms * mags
    else:
        a, gm, u, um = gate
        da = 1.13 * terms * gm + 2.0 ** -17 * np.abs(a) + 2.0 ** -60
        bound = da * np.abs(u) + (np.abs(a) + da) * terms * um
    bound = bound + ROUND[dtype] * (np.abs(exact) + bound) + (2.0 ** -24 if dtype == torch.float16 else 2.0 ** -126)
    got = got.double().cpu().numpy()
    assert got.shape == exact.shape
    worst = np.max(np.abs(got - exact) / bound) if got.size else 0.0
    assert worst <= 1.0, worst


def check(x, q, w, offsets, starts, alpha, act, out_dtype):
    """Runs the product (gated where act is given) and compares it."""
    X = x.double().cpu().numpy()
    K = X.shape[1]
    pre = alpha * ref.grouped(X, w, starts)
    mags = abs(alpha) * ref.grouped(np.abs(X), np.abs(w), starts)
    if act is None:
        got = ozk.mx4_gemv(x, q, offsets, alpha=alpha, out_dtype=out_dtype)
        near(got, pre, mags, K, got.dtype)
    else:
        H = w.shape[1] // 2
        got = ozk.mx4_gated_gemv(x, q, offsets, activation=act, alpha=alpha, out_dtype=out_dtype)
        a, u = act64(pre[:, :H], act), pre[:, H:]
        near(got, a * u, None, K, got.dtype, (a, mags[:, :H], u, mags[:, H:]))
    assert ozk.ozk_stream_status() == 0
    return got


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_plain(T, N, K, fmt, dtype):
    q, w = weights(N, K, fmt, 1, seed=N + K)
    x = normal(T, K, seed=T, dtype=dtype)
    check(x, q, w, None, [0, T], 0.5, None, torch.float32)
    check(x, q, w, None, [0, T], 1.0, None, None)


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated(T, N, K, fmt, act):
    q, w = weights(2 * N, K, fmt, 1, seed=N + K)
    dtype = torch.float16 if act == "gelu" else torch.bfloat16
    check(normal(T, K, seed=T, dtype=dtype), q, w, None, [0, T], 1.0 / math.sqrt(K), act, torch.float32)
    check(normal(T, K, seed=T, dtype=dtype), q, w, None, [0, T], 1.0 / math.sqrt(K), act, None)


@pytest.mark.parametrize("counts", [[0, 1, 0], [3, 0, 1, 20, 0, 2], [1] * 24, [0] * 40 + [5] + [0] * 30 + [9, 40]])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("act", [None, "silu"])
def test_grouped(counts, fmt, act):
    """Experts of 72 columns: their scale rows start inside a block of 128.  Rows in no group stay as they are."""
    starts = np.cumsum([2] + counts).tolist()
    T, K, N = starts[-1] + 3, 328, 72
    q, w = weights(N * (2 if act else 1), K, fmt, len(counts), seed=7)
    x = normal(T, K, seed=8, dtype=torch.bfloat16)
    offsets = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = torch.full((T, N), 77.0, dtype=torch.float32, device="cuda")
    if act:
        ozk.mx4_gated_gemv(x, q, offsets, alpha=0.1, out=out)
    else:
        ozk.mx4_gemv(x, q, offsets, alpha=0.1, out=out)
    inner = slice(starts[0], starts[-1])
    assert bool((out[: starts[0]] == 77).all()) and bool((out[starts[-1]:] == 77).all())
    X = x[inner].double().cpu().numpy()
    rel = [s - starts[0] for s in starts]
    pre, mags = 0.1 * ref.grouped(X, w, rel), 0.1 * ref.grouped(np.abs(X), np.abs(w), rel)
    if act:
        a, u = act64(pre[:, :N], act), pre[:, N:]
        near(out[inner], a * u, None, K, out.dtype, (a, mags[:, :N], u, mags[:, N:]))
    else:
        near(out[inner], pre, mags, K, out.dtype)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("bad", [[0, 9, 4, 6, 11], [-3, 2, 4, 6, 11], [0, 2, 4, 6, 12]])
def test_bad_offsets_are_cut_and_reported(bad):
    T, N, K, groups = 11, 48, 128, 4
    q, w = weights(N, K, "nvfp4", groups, seed=1)
    x = normal(T, K, seed=2, dtype=torch.bfloat16)
    got = ozk.mx4_gemv(x, q, torch.tensor(bad, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    cut = np.minimum(np.maximum.accumulate(np.maximum(bad, 0)), T).tolist()
    X = x.double().cpu().numpy()
    near(got[cut[0]: cut[-1]], ref.grouped(X, w, cut), ref.grouped(np.abs(X), np.abs(w), cut), K, got.dtype)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("T,N", [(1, 33), (2, 2600), (2, 5000), (2, 16000), (5, 33), (7, 2600), (7, 8200), (7, 16000), (12, 33),
                                 (12, 2600), (20, 8200)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_of_any_range(fmt, T, N):
    """Rows whose elements lie up to 2^226 apart, the large ones where the weights are zero: every element counts."""
    K = 700
    wide = normal(N, K, seed=3)
    wide[:, ::7] = 0.0
    q = ozk.mx4_quantize(wide, fmt)
    w = ozk.mx4_dequantize(q, torch.float64).cpu().numpy()[None]
    x = normal(T, K, seed=4)
    for t in range(T):
        if t % 5 == 0:
            x[t, ::7] = 2.0 ** 60
        if t % 5 == 1:
            x[t, 14::7] = 2.0 ** 127
        if t % 5 == 2:
            x[t] *= 2.0 ** -120
        if t % 5 == 3:
            x[t] *= 2.0 ** -100
            x[t, 630] = 2.0 ** 126  # in a later chunk than the first
    x = x.bfloat16()
    check(x, q, w, None, [0, T], 1.0, None, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_infinities_and_nans_stay_in_their_sums(fmt, dtype):
    T, N, K = 4, 40, 200
    wn = normal(N, K, seed=5)
    wn[11, 33] = float("nan")  # a block of NaNs in row 11
    wn[12, :96] = 0.0
    q = ozk.mx4_quantize(wn, fmt)
    w = ozk.mx4_dequantize(q, torch.float64)
    x = normal(T, K, seed=6, dtype=dtype)
    x[1, 50] = float("inf")
    x[2, 60] = float("nan")
    got = ozk.mx4_gemv(x, q, out_dtype=torch.float32).double()
    want = x.double() @ w.t()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    assert torch.allclose(got[fine], want[fine], rtol=1e-4, atol=1e-3)


def test_strides_and_alignment():
    """Rows of x on odd addresses and strides, a result with columns of its own around it."""
    T, N, K = 6, 100, 333
    q, w = weights(N, K, "nvfp4", 1, seed=9)
    big = normal(T, 3 * K + 2, seed=10, dtype=torch.bfloat16)
    x = big[:, 1: K + 1]
    X = x.double().cpu().numpy()
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        room = torch.full((T, N + 9), 5.0, dtype=dtype, device="cuda")
        out = room[:, 3: N + 3]
        assert ozk.mx4_gemv(x, q, out=out) is out
        near(out, ref.grouped(X, w, [0, T]), ref.grouped(np.abs(X), np.abs(w), [0, T]), K, dtype)
        assert bool((room[:, :3] == 5).all()) and bool((room[:, N + 3:] == 5).all())


def test_same_bits_every_time_and_in_a_graph():
    q, _ = weights(700, 1500, "nvfp4", 1, seed=11)
    x = normal(3, 1500, seed=12, dtype=torch.bfloat16)
    first = ozk.mx4_gemv(x, q)
    for _ in range(3):
        assert torch.equal(first, ozk.mx4_gemv(x, q))
    out = torch.empty_like(first)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ozk.mx4_gemv(x, q, out=out)
    again = normal(3, 1500, seed=13, dtype=torch.bfloat16)
    x.copy_(again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ozk.mx4_gemv(again, q))


def test_no_terms_and_no_rows():
    q = ozk.mx4_quantize(torch.empty(10, 0, device="cuda"))
    y = ozk.mx4_gemv(torch.empty(3, 0, dtype=torch.bfloat16, device="cuda"), q, alpha=float("inf"))
    assert y.shape == (3, 10) and not y.any()
    q, _ = weights(10, 64, "nvfp4", 1, seed=1)
    assert ozk.mx4_gemv(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), q).shape == (0, 10)


def test_refusals():
    q, _ = weights(10, 64, "nvfp4", 1, seed=1)
    x = normal(3, 64, seed=2, dtype=torch.bfloat16)
    grouped, _ = weights(10, 64, "nvfp4", 4, seed=1)
    offsets = torch.tensor([0, 1, 2, 3, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ozk.mx4_gemv(x[:, :60], q)
    with pytest.raises(ValueError):
        ozk.mx4_gemv(x, grouped)
    with pytest.raises(ValueError):
        ozk.mx4_gemv(x, grouped, offsets[:4].contiguous())
    with pytest.raises(ValueError):
        ozk.mx4_gemv(x.cpu(), q)
    with pytest.raises(ValueError):
        ozk.mx4_gated_gemv(x, q, activation="relu")
    with pytest.raises(ValueError):
        ozk.mx4_gated_gemv(x, weights(9, 64, "nvfp4", 1, seed=1)[0])
    with pytest.raises(ozk.OzkError):
        ozk.mx4_gemv(x.float(), q)
    with pytest.raises(TypeError):
        ozk.mx4_gemv(x, q, out_dtype=torch.int32)
    ozk.mx4_gemv(x, grouped, offsets)


def test_more_than_2_to_31_elements():
    """The last rows of a result past 2^31 elements are those of a call of their own."""
    T, N, K = 270400, 8000, 64
    q, _ = weights(N, K, "nvfp4", 1, seed=1)
    x = normal(T, K, seed=2, dtype=torch.bfloat16)
    y = ozk.mx4_gemv(x, q)
    assert torch.equal(y[-48:], ozk.mx4_gemv(x[-48:].clone(), q))
    assert ozk.ozk_stream_status() == 0


def test_calls_on_two_streams_at_once():
    q, _ = weights(3000, 2000, "mxfp4", 1, seed=3)
    xs = [normal(t, 2000, seed=t, dtype=torch.bfloat16) for t in (1, 2, 5, 12)]
    want = [ozk.mx4_gemv(x, q) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[ozk.mx4_gemv(x, q, stream=s) for x, s in zip(xs, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for row in got:
        for a, b in zip(row, want):
            assert torch.equal(a, b)
