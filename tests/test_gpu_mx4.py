"""Microscaled 4-bit matrices on the GPU: codes and scales bit for bit against
the 64-bit definition, and products against 64-bit products of the stored
values.

A product sums K terms in fp32; every one of its at most K additions is off by
at most 2^-23 of the magnitudes summed so far, so a result is within
K 2^-23 sum |a b| of the exact one, plus its own rounding; a 16-bit result is
the fp32 one rounded, bit for bit."""
import numpy as np
import pytest
import torch

import lowp_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
FORMATS = ["nvfp4", "mxfp4"]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def spread(rows, K, seed, dtype):
    """Values over many binades, so that scales differ from block to block."""
    g = gen(seed)
    x = torch.randn(rows, K, generator=g, device="cuda")
    e = torch.randint(-6, 7, (rows, -(-K // 16)), generator=g, device="cuda").repeat_interleave(16, dim=1)[:, :K]
    return torch.ldexp(x, e).to(dtype)


def check_quantized(q, x, prescale=1.0, starts=None):
    rows, K = x.shape
    starts = [0, rows] if starts is None else starts
    code, neg, byte = ref.quantize(x.double().cpu().numpy(), q.fmt, prescale)
    got_code, got_neg = ref.stored_codes(q.codes.cpu().numpy(), K)
    got_byte = ref.stored_scales(q.scales.cpu().numpy(), rows, K, q.fmt, starts)
    inside = np.arange(starts[0], starts[-1])
    assert np.array_equal(got_byte[inside], byte[inside])
    assert np.array_equal(got_code[inside], code[inside])
    kept = np.repeat(ref.scale_values(byte, q.fmt) > 0, ref.BLOCK[q.fmt], axis=1)[inside]
    assert np.array_equal((got_neg & (got_code > 0))[inside], (neg & (code > 0))[inside] & kept)
    v = ozk.mx4_dequantize(q, torch.float64).cpu().numpy()[inside]
    assert np.array_equal(v, ref.values(code, neg, byte, q.fmt, K)[inside], equal_nan=True)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 15), (3, 17), (2, 33), (33, 64), (129, 100), (5, 511), (4, 513),
                                    (1, 4096), (300, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.float64])
def test_quantize_bit_exact(fmt, rows, K, dtype):
    x = spread(rows, K, rows * 7 + K, dtype)
    check_quantized(ozk.mx4_quantize(x, fmt), x)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 6), (8, 8), (16, 48)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float64])
def test_quantize_any_alignment_and_stride(fmt, offset, pad, dtype):
    rows, K = 37, 290
    buf = torch.full((offset + rows * (K + pad) + 64,), float("nan"), device="cuda", dtype=dtype)
    x = buf[offset: offset + rows * (K + pad)].view(rows, K + pad)[:, :K]
    x.copy_(spread(rows, K, 5, dtype))
    q = ozk.mx4_quantize(x, fmt)
    check_quantized(q, x)
    out = torch.full((offset + rows * (K + pad) + 64,), 7.0, device="cuda", dtype=dtype)
    view = out[offset: offset + rows * (K + pad)].view(rows, K + pad)[:, :K]
    ozk.mx4_dequantize(q, out=view)
    assert torch.equal(view.double(), ozk.mx4_dequantize(q, torch.float64))
    view.fill_(7.0)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_edges(fmt):
    """Zeros, signed zeros, subnormals, the ends of the scales' ranges, Inf and NaN, each in blocks of their own."""
    tiny = float(np.float32(2.0 ** -149))
    blocks = [[0.0], [-0.0, 0.0], [tiny, -3 * tiny], [2.0 ** -126, -1.5 * 2.0 ** -127], [2.0 ** -130, 2.0 ** -128],
              [6 * 2.0 ** -10], [6 * 2.0 ** -10 * (1 + 2.0 ** -23)], [6 * 2.0 ** -9, 1e-3], [448 * 6.0, -448 * 5.0, 100.0],
              [3e38, -1e38, 1.0], [5000.0, 2688.0, 1344.0], [float("inf"), 1.0], [1.0, float("-inf")],
              [float("nan"), 2.0], [1.0], [2.0 - 2.0 ** -23], [2.0, 0.25, 0.26, -0.75, 1.25, 1.75, -2.5, 3.5]]
    x = torch.zeros(len(blocks), 96, device="cuda")
    for i, b in enumerate(blocks):
        x[i, 32: 32 + len(b)] = torch.tensor(b, dtype=torch.float64).float()
        x[i, 0] = 1.0  # the block before it
    check_quantized(ozk.mx4_quantize(x, fmt), x)


def test_quantize_ties_and_their_neighbours():
    """x' / s for every E4M3 scale s, at and next to every rounding boundary t s of the E2M1 codes, in fp32: the
    quotient's own rounding must not move any of them."""
    bounds = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in ref.E4M3[1:]:
        at = (bounds * s).astype(np.float32)
        for v in (at, np.nextafter(at, np.float32(np.inf)), np.nextafter(at, np.float32(0))):
            rows.append(np.concatenate(([6 * s], v, -v, [0.0])).astype(np.float32))
    x = torch.from_numpy(np.stack(rows)).cuda()
    check_quantized(ozk.mx4_quantize(x, "nvfp4"), x)
    # every bf16 magnitude below the top under every scale
    mags = torch.arange(0, 0x4500, 3, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    mags = mags[: mags.numel() // 15 * 15].view(-1, 15)
    for s in ref.E4M3[1::9]:
        x = torch.cat((torch.full((mags.size(0), 1), 6 * s, device="cuda", dtype=torch.bfloat16),
                       torch.minimum(mags, torch.tensor(6 * s, device="cuda", dtype=torch.bfloat16))), dim=1)
        check_quantized(ozk.mx4_quantize(x, "nvfp4"), x)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("prescale", [0.37, 2.0 ** 20, 1e-30])
def test_prescale(fmt, prescale):
    x = spread(9, 130, 3, torch.float32)
    check_quantized(ozk.mx4_quantize(x, fmt, prescale=prescale), x, prescale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_beyond_fp32_count_as_infinite(fmt):
    x = torch.ones(2, 64, device="cuda", dtype=torch.float64)
    x[0, 3] = 1e300
    check_quantized(ozk.mx4_quantize(x, fmt), x.float().double())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[0, 5, 0, 130, 1, 0], [128, 128], [127, 129, 300], [1] * 20])
def test_quantize_groups(fmt, counts):
    """Ragged groups, rows before the first and after the last left alone."""
    starts = (np.cumsum([0] + counts) + 3).tolist()
    rows, K = starts[-1] + 4, 200
    x = spread(rows, K, 11, torch.bfloat16)
    off = torch.tensor(starts, dtype=torch.int32, device="cuda")
    q = ozk.mx4_quantize(x, fmt, offsets=off)
    check_quantized(q, x, starts=starts)
    out = torch.full((rows, K), 9.0, device="cuda")
    ozk.mx4_dequantize(q, out=out)
    assert bool((out[:3] == 9).all()) and bool((out[starts[-1]:] == 9).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_equal_groups(fmt):
    w = spread(3 * 150, 192, 2, torch.bfloat16).view(3, 150, 192)
    check_quantized(ozk.mx4_quantize(w, fmt), w.view(450, 192), starts=[0, 150, 300, 450])
    wide = torch.zeros(3, 160, 200, device="cuda", dtype=torch.bfloat16)
    wide[:, :150, :192] = w
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = ozk.mx4_quantize(wide[:, :150, :192], fmt, stream=s)
    s.synchronize()
    check_quantized(q, w.view(450, 192), starts=[0, 150, 300, 450])


def check_product(c, a, b, alpha, K):
    """The fp32 product c against alpha a b^T of the stored values in 64 bits."""
    exact = alpha * (a @ b.t())
    mags = abs(alpha) * (a.abs() @ b.abs().t())
    err = (c.double() - exact).abs()
    assert bool((err <= K * 2.0 ** -23 * mags + 2.0 ** -24 * exact.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 64), (7, 300, 129), (16, 1024, 4096), (129, 257, 65),
                                   (300, 130, 513), (1000, 1537, 700), (513, 2050, 1088), (2300, 2100, 320)])
@pytest.mark.parametrize("dtype", TYPES)
def test_product(fmt, M, N, K, dtype):
    qa, qb = ozk.mx4_quantize(spread(M, K, 1, torch.bfloat16), fmt), ozk.mx4_quantize(spread(N, K, 2, torch.bfloat16), fmt)
    a, b = ozk.mx4_dequantize(qa, torch.float64), ozk.mx4_dequantize(qb, torch.float64)
    c = ozk.mx4_gemm(qa, qb, alpha=1.0 / 512, out_dtype=dtype)
    assert c.dtype == dtype and c.shape == (M, N)
    c32 = ozk.mx4_gemm(qa, qb, alpha=1.0 / 512, out_dtype=torch.float32)
    check_product(c32, a, b, 1.0 / 512, K)
    assert torch.equal(c, c32.to(dtype))
    assert torch.equal(c, ozk.mx4_gemm(qa, qb, alpha=1.0 / 512, out_dtype=dtype))  # the same bits again
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tiles_per_cta_exact(fmt):
    """Small whole numbers, exact in fp32: every output of many waves of tiles (both accumulators, reused stages)."""
    M, N, K = 5000, 6000, 576
    g = gen(4)
    a = torch.randint(-3, 4, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-3, 4, (N, K), generator=g, device="cuda").float()
    a[:, ::16] = 6.0  # scale 1 in every block (and 2^0 in mxfp4)
    b[:, ::16] = -6.0
    qa, qb = ozk.mx4_quantize(a, fmt), ozk.mx4_quantize(b, fmt)
    assert torch.equal(ozk.mx4_dequantize(qa), a) and torch.equal(ozk.mx4_dequantize(qb), b)
    want = (a.double() @ b.double().t())
    assert torch.equal(ozk.mx4_gemm(qa, qb, out_dtype=torch.float32).double(), want)
    assert torch.equal(ozk.mx4_gemm(qa, qb), want.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset,pad", [(0, 0), (0, 8), (1, 0), (4, 3), (8, 16)])
def test_product_output_alignment(dtype, offset, pad):
    M, N, K = 70, 200, 128
    qa, qb = ozk.mx4_quantize(spread(M, K, 1, torch.bfloat16)), ozk.mx4_quantize(spread(N, K, 2, torch.bfloat16))
    buf = torch.full((offset + M * (N + pad) + 32,), 7.0, device="cuda", dtype=dtype)
    view = buf[offset: offset + M * (N + pad)].view(M, N + pad)[:, :N]
    ozk.mx4_gemm(qa, qb, out=view)
    assert torch.equal(view, ozk.mx4_gemm(qa, qb, out_dtype=dtype))
    view.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_stays_in_its_row_and_column(fmt):
    M, N, K = 40, 300, 128
    x, w = spread(M, K, 1, torch.bfloat16), spread(N, K, 2, torch.bfloat16)
    clean = ozk.mx4_gemm(ozk.mx4_quantize(x, fmt), ozk.mx4_quantize(w, fmt))
    x[3, 5], w[290, 100] = float("nan"), float("inf")
    c = ozk.mx4_gemm(ozk.mx4_quantize(x, fmt), ozk.mx4_quantize(w, fmt))
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3, :] = True
    bad[:, 290] = True
    assert torch.equal(c.isnan(), bad)
    assert torch.equal(c[~bad], clean[~bad])


def test_empty_products():
    q = ozk.mx4_quantize(torch.empty(0, 64, device="cuda"))
    w = ozk.mx4_quantize(torch.ones(5, 64, device="cuda"))
    assert ozk.mx4_gemm(q, w).shape == (0, 5) and ozk.mx4_gemm(w, q).shape == (5, 0)
    e = ozk.mx4_quantize(torch.empty(5, 0, device="cuda"))
    assert torch.equal(ozk.mx4_gemm(e, e, out_dtype=torch.float32), torch.zeros(5, 5, device="cuda"))
    assert ozk.mx4_dequantize(e).shape == (5, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,N,K", [([3], 128, 64), ([0, 40, 1, 0, 200, 129], 300, 200), ([1] * 32, 256, 1024),
                                        ([500, 0, 700, 3], 520, 320), ([0, 0, 2], 64, 4096)])
def test_grouped_product(fmt, counts, N, K):
    starts, G = np.cumsum([0] + counts).tolist(), len(counts)
    T = starts[-1]
    off = torch.tensor(starts, dtype=torch.int32, device="cuda")
    qx = ozk.mx4_quantize(spread(T, K, 1, torch.bfloat16), fmt, offsets=off)
    qw = ozk.mx4_quantize(spread(G * N, K, 2, torch.bfloat16).view(G, N, K), fmt)
    x, w = ozk.mx4_dequantize(qx, torch.float64), ozk.mx4_dequantize(qw, torch.float64).view(G, N, K)
    y = ozk.mx4_grouped_gemm(qx, qw, alpha=0.01, out_dtype=torch.float32)
    for g in range(G):
        rows = slice(starts[g], starts[g + 1])
        check_product(y[rows], x[rows], w[g], float(np.float32(0.01)), K)
    for dtype in TYPES:
        assert torch.equal(ozk.mx4_grouped_gemm(qx, qw, alpha=0.01, out_dtype=dtype), y.to(dtype))
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_grouped_product_of_some_rows(fmt):
    """Groups that start after the first row, inside a row block of scales, and end before the last."""
    starts, T, N, K = [133, 140, 140, 300, 301], 330, 200, 192
    G, off = 4, torch.tensor(starts, dtype=torch.int32, device="cuda")
    qx = ozk.mx4_quantize(spread(T, K, 1, torch.bfloat16), fmt, offsets=off)
    qw = ozk.mx4_quantize(spread(G * N, K, 2, torch.bfloat16).view(G, N, K), fmt)
    x = torch.zeros(T, K, device="cuda", dtype=torch.float64)
    ozk.mx4_dequantize(qx, out=x)
    w = ozk.mx4_dequantize(qw, torch.float64).view(G, N, K)
    y = torch.full((T, N), 5.0, device="cuda")
    ozk.mx4_grouped_gemm(qx, qw, out=y)
    for g in range(G):
        rows = slice(starts[g], starts[g + 1])
        check_product(y[rows], x[rows], w[g], 1.0, K)
    assert bool((y[:133] == 5).all()) and bool((y[301:] == 5).all())
    assert ozk.ozk_stream_status() == 0


def test_results_past_32_bits():
    """An output of more than 2^31 elements, and codes and weights whose last rows lie past 2^31 bytes."""
    M, N, K = 300_000, 7200, 128
    qb = ozk.mx4_quantize(spread(N, K, 2, torch.bfloat16))
    qa = ozk.mx4_quantize(spread(1000, K, 1, torch.bfloat16).repeat(300, 1))
    c = ozk.mx4_gemm(qa, qb)
    assert torch.equal(c[-1000:], c[:1000])
    small = ozk.mx4_gemm(ozk.mx4_quantize(spread(1000, K, 1, torch.bfloat16)), qb)
    assert torch.equal(c[:1000], small)
    del c
    G, N, K = 40, 16384, 8192  # codes: 2.7 GB
    w = spread(N, K, 3, torch.bfloat16).repeat(G, 1).view(G, N, K)
    qw = ozk.mx4_quantize(w)
    del w
    off = torch.arange(G + 1, dtype=torch.int32, device="cuda") * 2
    x = spread(2, K, 4, torch.bfloat16).repeat(G, 1)
    y = ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, offsets=off), qw, out_dtype=torch.float32)
    assert torch.equal(y[-2:], y[:2]) and bool((y[:2] != 0).any())


def test_other_streams_and_graphs():
    fmt = "nvfp4"
    G, N, K, T = 3, 256, 512, 12
    w = ozk.mx4_quantize(spread(G * N, K, 2, torch.bfloat16).view(G, N, K), fmt)
    x = spread(T, K, 1, torch.bfloat16)
    off = torch.tensor([0, 3, 3, 12], dtype=torch.int32, device="cuda")
    want = ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, fmt, offsets=off), w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, fmt, offsets=off, stream=s), w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, fmt, offsets=off), w)
    x.copy_(spread(T, K, 9, torch.bfloat16))
    off.copy_(torch.tensor([0, 0, 7, 12], dtype=torch.int32))
    graph.replay()
    want = ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, fmt, offsets=off), w)
    assert torch.equal(y, want)


def test_quantize_then_product_back_to_back():
    """Calls on one stream that reuse memory at once: each waits for the one before it."""
    K = 1024
    ws = [ozk.mx4_quantize(spread(640, K, 30 + i, torch.bfloat16)) for i in range(3)]
    xs = [spread(96, K, 40 + i, torch.bfloat16) for i in range(6)]
    want = [ozk.mx4_gemm(ozk.mx4_quantize(x), ws[i % 3]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    buf = torch.empty_like(xs[0])
    got = []
    for i, x in enumerate(xs):
        buf.copy_(x)
        got.append(ozk.mx4_gemm(ozk.mx4_quantize(buf), ws[i % 3]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_wrapper_refusals():
    x = torch.ones(8, 64, device="cuda")
    with pytest.raises(ValueError):
        ozk.mx4_quantize(x, "fp4")
    with pytest.raises(ValueError):
        ozk.mx4_quantize(x.t())
    with pytest.raises(ValueError):
        ozk.mx4_quantize(x[:1].expand(8, 64))
    with pytest.raises(ValueError):
        ozk.mx4_quantize(x.cpu())
    with pytest.raises(TypeError):
        ozk.mx4_quantize(x.int())
    with pytest.raises(TypeError):
        ozk.mx4_quantize(x, offsets=torch.tensor([0, 8], device="cuda"))  # int64
    with pytest.raises(ozk.OzkError):
        ozk.mx4_quantize(x, prescale=0.0)
    a, b = ozk.mx4_quantize(x), ozk.mx4_quantize(x, "mxfp4")
    with pytest.raises(ValueError):
        ozk.mx4_gemm(a, b)
    with pytest.raises(ozk.OzkError):
        ozk.mx4_gemm(a, a, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        ozk.mx4_gemm(a, a, out=torch.empty(8, 9, device="cuda"))
    with pytest.raises(ValueError):
        ozk.mx4_grouped_gemm(a, a)
    with pytest.raises(ValueError):
        ozk.Mx4(a.codes[:, :16], a.scales, 8, 64, "nvfp4")
