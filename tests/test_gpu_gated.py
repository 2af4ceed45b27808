"""Gated products of rows grouped by expert on the GPU, their slopes and their
gradients, against 64-bit forms (gated_reference has the bounds)."""
import math

import numpy as np
import pytest
import torch

import gated_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}
# rows of each group, H, K
SHAPES = [([1], 1, 8), ([1], 8, 8), ([5, 0, 17], 64, 64), ([130, 3, 0, 64], 136, 264), ([300, 1], 36, 1032), ([1] * 24, 256, 512),
          ([16, 15, 0, 0, 49, 128, 129], 200, 136), ([700, 0, 260], 296, 520), ([61] * 30, 264, 520), ([2000], 513, 200),
          ([900, 1100], 1040, 1000)]


def normal(*shape, seed, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def setup(counts, H, K, dtype, before=0, after=0):
    starts = np.cumsum([before] + counts).tolist()
    x = normal(starts[-1] + after, K, seed=1, dtype=dtype)
    w = (normal(len(counts), 2 * H, K, seed=2, dtype=torch.float32) / math.sqrt(K)).to(dtype)
    return x, w, torch.tensor(starts, dtype=torch.int32, device="cuda"), starts


def wide(t):
    return t.detach().double().cpu().numpy()


def near(got, exact, bound, dtype, extra=0.0):
    assert got.dtype == dtype and tuple(got.shape) == exact.shape
    limit = ref.rounded(bound, exact, HALF[dtype], LEAST[dtype]) + extra
    worst = np.max(np.abs(wide(got) - exact) / limit) if exact.size else 0.0
    assert worst <= 1.0, worst


@pytest.mark.parametrize("counts,H,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ref.ACTS)
def test_product_and_slopes(counts, H, K, dtype, act):
    x, w, offsets, starts = setup(counts, H, K, dtype)
    slopes = torch.empty(2, x.shape[0], H, device="cuda")
    h = ozk.grouped_gated_gemm(x, w, offsets, activation=act, slopes=slopes)
    assert torch.equal(h, ozk.grouped_gated_gemm(x, w, offsets, activation=act))  # the same with and without slopes
    X, W = wide(x), wide(w)
    for g, (a, b) in enumerate(zip(starts, starts[1:])):
        r = ref.Gated(X[a:b], W[g], act)
        near(h[a:b], r.h, r.dh, dtype)
        near(slopes[0, a:b], r.by_gate, r.d_gate, torch.float32)
        near(slopes[1, a:b], r.by_up, r.d_up, torch.float32)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("counts,H,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients(counts, H, K, dtype, act):
    """The slopes are in fp32, the gradient of the projections is rounded to fp32 and to 16 bits; a rounding is off by at
    most half a step of its value, and the products sum 2 H (rows of the group) terms in fp32."""
    x, w, offsets, starts = setup(counts, H, K, dtype)
    dh = normal(x.shape[0], H, seed=3, dtype=dtype)
    x.requires_grad_(), w.requires_grad_()
    h = ozk.grouped_gated_gemm(x, w, offsets, activation=act)
    assert h.requires_grad
    dx, dw = torch.autograd.grad(h, (x, w), dh)
    X, W, D = wide(x), wide(w), wide(dh)
    for g, (a, b) in enumerate(zip(starts, starts[1:])):
        r = ref.Gated(X[a:b], W[g], act)
        pre = np.concatenate((D[a:b] * r.by_gate, D[a:b] * r.by_up), axis=1)
        err = np.concatenate([np.abs(D[a:b]) * ref.rounded(e, v, 2.0 ** -23, 2.0 ** -126)
                              for v, e in ((r.by_gate, r.d_gate), (r.by_up, r.d_up))], axis=1)
        err = ref.rounded(err, pre, HALF[dtype], LEAST[dtype])
        mags = np.abs(pre) + err
        near(dx[a:b], pre @ W[g], err @ np.abs(W[g]) + 2 * H * 2.0 ** -23 * (mags @ np.abs(W[g])), dtype)
        near(dw[g], pre.T @ X[a:b], err.T @ np.abs(X[a:b]) + (b - a) * 2.0 ** -23 * (mags.T @ np.abs(X[a:b])), dtype)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("H", [64, 61])
def test_rows_in_no_group(H):
    """They stay as they are, and have no gradient."""
    x, w, offsets, starts = setup([9, 0, 40], H, 72, torch.bfloat16, before=3, after=6)
    T, inner = x.shape[0], slice(starts[0], starts[-1])
    out = torch.full((T, H), 7.0, dtype=x.dtype, device="cuda")
    slopes = torch.full((2, T, H), 7.0, device="cuda")
    ozk.grouped_gated_gemm(x, w, offsets, out=out, slopes=slopes)
    dpre = torch.full((T, 2 * H), 7.0, dtype=x.dtype, device="cuda")
    dh = normal(T, H, seed=3, dtype=x.dtype)
    ozk.gated_grad(dh, slopes, offsets, out=dpre)
    for t in (out, slopes[0], slopes[1], dpre):
        assert bool((t[: starts[0]] == 7).all()) and bool((t[starts[-1]:] == 7).all()) and not bool((t[inner] == 7).all())
    for half in range(2):
        want = (dh[inner].float() * slopes[half, inner]).to(x.dtype)  # rounded to fp32 and to 16 bits
        assert torch.equal(dpre[inner, half * H: half * H + H], want)
    x.requires_grad_()
    h = ozk.grouped_gated_gemm(x, w, offsets)
    h.backward(dh)
    assert not x.grad[: starts[0]].any() and not x.grad[starts[-1]:].any() and x.grad[inner].any()
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 1024), (17, 1032), (300, 2056)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gated_grad_alone(T, H, dtype):
    """Products rounded to fp32 and to 16 bits; any alignment."""
    slopes, d16 = normal(2, T, H, seed=4, dtype=torch.float32), normal(T, H, seed=5, dtype=dtype)
    want = torch.cat((d16.float() * slopes[0], d16.float() * slopes[1]), dim=1).to(dtype)
    assert torch.equal(ozk.gated_grad(d16, slopes), want)
    room = torch.full((T, 2 * H + 3), 9.0, dtype=dtype, device="cuda")
    odd = torch.empty(2, T, H + 5, device="cuda")[:, :, 3: H + 3]
    odd.copy_(slopes)
    ozk.gated_grad(d16, odd, out=room[:, 1: 2 * H + 1])
    assert torch.equal(room[:, 1: 2 * H + 1], want) and bool((room[:, 0] == 9).all()) and bool((room[:, 2 * H + 1:] == 9).all())
    one = torch.ones((), dtype=dtype, device="cuda").expand(T, H)
    assert torch.equal(ozk.gated_grad(one, slopes), torch.cat((slopes[0], slopes[1]), dim=1).to(dtype))


def test_results_beside_others():
    """A result and slopes with rows of odd length: nothing beside them is touched."""
    x, w, offsets, starts = setup([70, 30], 40, 64, torch.bfloat16)
    want = ozk.grouped_gated_gemm(x, w, offsets)
    for left in (0, 3, 8):
        room = torch.full((100, 40 + left + 5), 9.0, dtype=x.dtype, device="cuda")
        sroom = torch.full((2, 100, 40 + left + 8), 9.0, device="cuda")
        ozk.grouped_gated_gemm(x, w, offsets, out=room[:, left: left + 40], slopes=sroom[:, :, left: left + 40])
        assert torch.equal(room[:, left: left + 40], want)
        for t in (room, sroom[0], sroom[1]):
            assert bool((t[:, :left] == 9).all()) and bool((t[:, left + 40:] == 9).all())


def test_no_terms():
    x = torch.empty(4, 0, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(2, 16, 0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    slopes = torch.full((2, 4, 8), 9.0, device="cuda")
    assert not ozk.grouped_gated_gemm(x, w, offsets, slopes=slopes).any() and not slopes.any()


def test_a_nan_stays_in_its_row_and_column():
    x, w, offsets, starts = setup([40, 40], 72, 80, torch.bfloat16)
    x[5, 3] = float("nan")
    w[1, 10, 7] = float("nan")
    w[1, 72 + 11, 7] = float("inf")
    x[40:, 7] = 1.0
    h = ozk.grouped_gated_gemm(x, w, offsets)
    bad = ~torch.isfinite(h)
    want = torch.zeros_like(bad)
    want[5] = True
    want[40:, 10:12] = True
    assert torch.equal(bad, want)


def test_bad_offsets_are_cut_and_reported():
    x, w, _, _ = setup([10, 10, 10], 64, 64, torch.bfloat16)
    bad = torch.tensor([0, 20, 5, 40], dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, 20, 20, 30], dtype=torch.int32, device="cuda")
    got = ozk.grouped_gated_gemm(x, w, bad)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    assert torch.equal(got, ozk.grouped_gated_gemm(x, w, cut))
    slopes, dh = normal(2, 30, 64, seed=1, dtype=torch.float32), normal(30, 64, seed=2, dtype=x.dtype)
    assert torch.equal(ozk.gated_grad(dh, slopes, bad), ozk.gated_grad(dh, slopes))
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_INVALID_ARG
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("pairs,cta", [(0, 0), (1, 0), (1, 1)])
def test_a_withheld_copy_ends_the_call(pairs, cta):
    """The failure path of the products: the wait runs out, the kernel returns, the status says so."""
    x, w, offsets, _ = setup([600], 256, 512, torch.bfloat16)
    want = ozk.grouped_gated_gemm(x, w, offsets)
    ozk.ozk_withhold_next_product(pairs, cta, 3, 20000)
    ozk.grouped_gated_gemm(x, w, offsets)
    assert ozk.ozk_stream_status() == ozk.OZK_ERR_TIMEOUT
    assert torch.equal(ozk.grouped_gated_gemm(x, w, offsets), want)
    assert ozk.ozk_stream_status() == 0


def test_only_what_is_asked_for():
    x, w, offsets, _ = setup([10, 6], 32, 64, torch.bfloat16)
    dh = normal(16, 32, seed=3, dtype=x.dtype)
    both = torch.autograd.grad(ozk.grouped_gated_gemm(x.requires_grad_(), w.requires_grad_(), offsets), (x, w), dh)
    for only in (0, 1):
        a, b = x.detach().requires_grad_(only == 0), w.detach().requires_grad_(only == 1)
        ozk.grouped_gated_gemm(a, b, offsets).backward(dh)
        assert torch.equal((a, b)[only].grad, both[only]) and (a, b)[1 - only].grad is None
    with torch.no_grad():
        assert not ozk.grouped_gated_gemm(x, w, offsets).requires_grad
    g, = torch.autograd.grad(ozk.grouped_gated_gemm(x, w, offsets).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), w)


def test_replayed_with_other_rows():
    """A captured graph of the product and its gradients, replayed with other values and offsets."""
    x, w, offsets, _ = setup([50, 14], 72, 136, torch.bfloat16)
    dh = normal(64, 72, seed=3, dtype=x.dtype)
    slopes = torch.empty(2, 64, 72, device="cuda")

    def step():
        h = ozk.grouped_gated_gemm(x, w, offsets, slopes=slopes)
        dpre = ozk.gated_grad(dh, slopes, offsets)
        return h, ozk.grouped_gemm_dx(dpre, w, offsets), ozk.grouped_gemm_dw(dpre, x, offsets)

    step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    x.copy_(normal(64, 136, seed=9, dtype=x.dtype))
    offsets.copy_(torch.tensor([0, 7, 64], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, step()):
        assert torch.equal(a, b)
    assert ozk.ozk_stream_status() == 0


def test_on_another_stream():
    x, w, offsets, _ = setup([300, 200], 128, 256, torch.bfloat16)
    want = ozk.grouped_gated_gemm(x, w, offsets)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ozk.grouped_gated_gemm(x, w, offsets, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    x, w, offsets, _ = setup([10, 6], 32, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm(x, w, offsets, activation="relu")
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm(x, w[:, :63], offsets)
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm(x[:, :56], w, offsets)
    with pytest.raises(TypeError):
        ozk.grouped_gated_gemm(x.half(), w, offsets)
    with pytest.raises(TypeError):
        ozk.grouped_gated_gemm(x, w, offsets, slopes=torch.empty(2, 16, 32, dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm(x, w, offsets, slopes=torch.empty(2, 16, 31, device="cuda"))
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm(x, w, offsets[:2].contiguous())
    slopes = torch.empty(2, 16, 32, device="cuda")
    with pytest.raises(ValueError):
        ozk.gated_grad(torch.empty(16, 31, dtype=x.dtype, device="cuda"), slopes)
    with pytest.raises(ValueError):
        ozk.gated_grad(torch.empty(16, 32, dtype=x.dtype), slopes)
    with pytest.raises(ozk.OzkError):
        ozk.gated_grad(slopes[0], slopes)  # a gradient in fp32
    with pytest.raises(ozk.OzkError):  # a result over the slopes
        ozk.gated_grad(x[:, :32], slopes, out=slopes.view(x.dtype)[0, :, :].view(16, 64))


@pytest.mark.parametrize("H,K", [(61, 72), (64, 40)])
def test_backward_pass_in_one_call(H, K):
    """It is gated_grad and both products, with zeros where a row has no group and a group no rows; what is not asked
    for is not computed."""
    x, w, offsets, starts = setup([9, 0, 40], H, K, torch.bfloat16, before=3, after=6)
    T = x.shape[0]
    slopes = normal(2, T, H, seed=4, dtype=torch.float32)
    dh = normal(T, H, seed=3, dtype=x.dtype)
    torch.full((1 << 18,), float("nan"), device="cuda", dtype=torch.bfloat16)  # what unwritten memory would hold
    room = torch.zeros(T, -(-2 * H // 8) * 8, dtype=x.dtype, device="cuda")
    dpre = ozk.gated_grad(dh, slopes, offsets, out=room[:, : 2 * H])
    want_x = ozk.grouped_gemm_dx(dpre, w, offsets, out=torch.zeros(T, K, dtype=x.dtype, device="cuda"))
    want_w = ozk.grouped_gemm_dw(dpre, x, offsets)
    dx, dw = ozk.grouped_gated_gemm_grad(dh.float(), x, w, offsets, slopes)  # rounded to bf16 again
    assert torch.equal(dx, want_x) and torch.equal(dw, want_w) and not dw[1].any()
    assert ozk.grouped_gated_gemm_grad(dh, x, w, offsets, slopes, need_dw=False)[1] is None
    dx, dw = ozk.grouped_gated_gemm_grad(dh, x, w, offsets, slopes, need_dx=False)
    assert dx is None and torch.equal(dw, want_w)
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm_grad(dh[:, :H - 1], x, w, offsets, slopes)
    with pytest.raises(ValueError):
        ozk.grouped_gated_gemm_grad(dh, x, w, offsets, slopes[:, :, : H - 1])
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("act", ref.ACTS)
def test_far_arguments(act):
    """Far to the right the activation is g with slope 1, far to the left 0 with slope 0, also where g^2 leaves fp32."""
    g = [1e3, 1e10, 3e19, 1e30, -1e3, -1e10, -3e19, -1e30]
    x = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor(g)
    x[:, 1] = 1.0
    w = torch.zeros(1, 2, 8, dtype=torch.bfloat16, device="cuda")
    w[0, 0, 0] = w[0, 1, 1] = 1.0  # g is the first element, u is 1
    offsets = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    slopes = torch.empty(2, 8, 1, device="cuda")
    h = ozk.grouped_gated_gemm(x, w, offsets, activation=act, slopes=slopes)
    want = torch.clamp(x[:, 0], min=0.0)
    assert torch.equal(h[:, 0], want) and torch.equal(slopes[1, :, 0], want.float())
    assert torch.equal(slopes[0, :, 0], (x[:, 0] > 0).float())


@pytest.mark.parametrize("H,K,T", [(0, 16, 5), (8, 16, 0), (0, 16, 0)])
def test_nothing_to_multiply(H, K, T):
    """No columns or no rows: empty results, gradients of zeros."""
    x = torch.ones(T, K, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.ones(2, 2 * H, K, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    offsets = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
    h = ozk.grouped_gated_gemm(x, w, offsets)
    assert h.shape == (T, H)
    dx, dw = torch.autograd.grad(h, (x, w), torch.ones_like(h))
    assert dx.shape == x.shape and not dx.any() and dw.shape == w.shape and not dw.any()
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("act", ref.ACTS)
def test_the_activation_itself(act):
    """The second slope is act(g) in fp32, the first act'(g) where u is 1: at every fp16 value of g from -8 to 8.  Off by
    off(g) of act(g) (gated_reference).  act' = P + g P' has terms of at most 1 and 1.2, in silu's and gelu_tanh's case
    g P (1 - P) z', where 1 - P may be off by all of P's error: off(g) P (1 + 2 |g| z') together, below 64 units times 8
    where P is not tiny (|z| <= 19), and nothing elsewhere."""
    g = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.float16)
    g = g[torch.isfinite(g) & (g.abs() <= 8)]
    x = torch.zeros(g.numel(), 8, dtype=torch.float16, device="cuda")
    x[:, 0], x[:, 1] = g, 1.0
    w = torch.zeros(1, 2, 8, dtype=torch.float16, device="cuda")
    w[0, 0, 0] = w[0, 1, 1] = 1.0
    offsets = torch.tensor([0, g.numel()], dtype=torch.int32, device="cuda")
    slopes = torch.empty(2, g.numel(), 1, device="cuda")
    ozk.grouped_gated_gemm(x, w, offsets, activation=act, slopes=slopes)
    value, slope = ref.act(wide(g), act)
    tail = np.array([math.erfc(-v * math.sqrt(0.5)) / 2 for v in wide(g)]) if act == "gelu" else None
    if tail is not None:  # 1 + erf loses the tail's digits to 64 bits
        value = wide(g) * tail
    assert np.all(np.abs(wide(slopes[1, :, 0]) - value) <= ref.off(wide(g), act) * np.abs(value) + 2.0 ** -140)
    assert np.all(np.abs(wide(slopes[0, :, 0]) - slope) <= 64 * 2.0 ** -23 * 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_operands_in_padded_buffers(dtype):
    """Rows of 60 columns in buffers of 72, groups apart: the same bits as tight ones of 64 with zeros, gradients too."""
    x, w, offsets, _ = setup([33, 0, 100], 40, 60, dtype)
    T = x.shape[0]
    xs, ws = torch.full((T, 72), 9.0, dtype=dtype, device="cuda"), torch.full((3, 85, 72), 9.0, dtype=dtype, device="cuda")
    xs[:, :60], ws[:, :80, :60] = x, w
    xz, wz = torch.zeros(T, 64, dtype=dtype, device="cuda"), torch.zeros(3, 80, 64, dtype=dtype, device="cuda")
    xz[:, :60], wz[..., :60] = x, w
    dh = normal(T, 40, seed=3, dtype=dtype)
    results = []
    for a, b in ((xs[:, :60], ws[:, :80, :60]), (xz, wz)):
        a, b = a.detach().requires_grad_(), b.detach().requires_grad_()
        h = ozk.grouped_gated_gemm(a, b, offsets, activation="gelu")
        dx, dw = torch.autograd.grad(h, (a, b), dh)
        results.append((h.detach(), dx[:, :60], dw[..., :60]))
    for got, want in zip(*results):
        assert torch.equal(got, want)


@pytest.mark.parametrize("how", ["expanded", "transposed", "double"])
def test_gradients_that_come_in_other_forms(how):
    x, w, offsets, _ = setup([20, 13], 24, 40, torch.bfloat16)
    x.requires_grad_(), w.requires_grad_()
    if how == "expanded":
        dh = torch.ones((), dtype=x.dtype, device="cuda").expand(33, 24)
    elif how == "transposed":
        dh = normal(24, 33, seed=3, dtype=x.dtype).t()
    else:
        dh = normal(33, 24, seed=3, dtype=x.dtype)
    h = ozk.grouped_gated_gemm(x, w, offsets)
    want = torch.autograd.grad(h, (x, w), dh.contiguous(), retain_graph=True)
    if how == "double":
        got = torch.autograd.grad(h.double(), (x, w), dh.double())
    else:
        got = torch.autograd.grad(h, (x, w), dh)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_training_step_in_a_graph():
    """Forward and backward through autograd, captured and replayed with other values.  (With an eager graph of the same
    leaves alive autograd refuses the capture, whatever the function.)"""
    x, w, offsets, _ = setup([50, 14], 72, 136, torch.bfloat16)
    dh = normal(64, 72, seed=3, dtype=x.dtype)
    x.requires_grad_(), w.requires_grad_()

    def step():
        h = ozk.grouped_gated_gemm(x, w, offsets)
        return (h, *torch.autograd.grad(h, (x, w), dh))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    with torch.no_grad():
        dh.copy_(normal(64, 72, seed=4, dtype=x.dtype))
        offsets.copy_(torch.tensor([0, 7, 64], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, step()):
        assert torch.equal(a.detach(), b.detach())
    assert ozk.ozk_stream_status() == 0


def test_more_than_2_to_31_elements():
    """Results, slopes and gradients past 2^31 elements, where the last rows are those of a call of their own."""
    T, H, K = 270400, 8000, 8
    x = normal(T, K, seed=1, dtype=torch.bfloat16)
    w = normal(1, 2 * H, K, seed=2, dtype=torch.bfloat16)
    last = slice(T - 40, T)
    slopes = torch.empty(2, T, H, device="cuda")
    h = ozk.grouped_gated_gemm(x, w, torch.tensor([0, T], dtype=torch.int32, device="cuda"), slopes=slopes)
    few = torch.empty(2, 40, H, device="cuda")
    want = ozk.grouped_gated_gemm(x[last].clone(), w, torch.tensor([0, 40], dtype=torch.int32, device="cuda"), slopes=few)
    assert torch.equal(h[last], want) and torch.equal(slopes[:, last], few)
    dpre = ozk.gated_grad(h, slopes)
    assert torch.equal(dpre[last], ozk.gated_grad(want, few))
    assert ozk.ozk_stream_status() == 0
