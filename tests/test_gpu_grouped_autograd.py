"""Gradients of ozk.grouped_gemm through autograd, on small whole numbers: every sum is exact, so they equal those of the
64-bit form."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu


def whole(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)


def padded(t):
    """A view of t's values with rows 16 bytes apart in multiples (buffers of 64 columns)."""
    buf = torch.zeros(*t.shape[:-1], 64, device="cuda", dtype=t.dtype)
    buf[..., : t.shape[-1]] = t
    return buf[..., : t.shape[-1]]


def plain(x, w, starts):
    """The product in 64 bits, zeros for rows in no group."""
    y = torch.zeros(x.size(0), w.size(1), device="cuda", dtype=torch.float64)
    parts = [x[a:b] @ w[g].t() for g, (a, b) in enumerate(zip(starts, starts[1:]))]
    return torch.cat([y[: starts[0]], *parts, y[starts[-1]:]])


def case(N=24, K=40, dtype=torch.bfloat16, starts=(0, 5, 5, 19, 20)):
    starts = list(starts)
    T, G = starts[-1], len(starts) - 1
    x, w = whole(T, K, seed=1, dtype=dtype), whole(G, N, K, seed=2, dtype=dtype)
    if K % 8:
        x, w = padded(x), padded(w)
    return x, w, torch.tensor(starts, dtype=torch.int32, device="cuda"), starts


def check(x, w, off, starts, weight, out_dtype=None):
    """Gradients of sum(weight * y)."""
    x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    y = ozk.grouped_gemm(x, w, off, out_dtype=out_dtype)
    assert y.requires_grad and y.dtype == (out_dtype or x.dtype)
    inside = slice(starts[0], starts[-1])
    (y[inside] * weight[inside].to(y.dtype)).sum().backward()
    hx, hw = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    want = plain(hx, hw, starts)
    assert torch.equal(y.detach()[inside].double(), want.detach()[inside])
    (want[inside] * weight[inside].double()).sum().backward()
    assert torch.equal(x.grad.double(), hx.grad) and torch.equal(w.grad.double(), hw.grad)
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("N,K", [(24, 40), (13, 40), (24, 60), (1, 8)])
def test_gradients(N, K, out_dtype, dtype):
    """N of any size: the result's gradient comes with rows that bulk copies cannot read."""
    x, w, off, starts = case(N, K, dtype)
    check(x, w, off, starts, whole(x.size(0), N, seed=3, dtype=dtype), out_dtype)


def test_gradient_of_a_plain_sum():
    """It comes as one number expanded to the result's shape."""
    x, w, off, starts = case()
    x, w = x.requires_grad_(), w.requires_grad_()
    ozk.grouped_gemm(x, w, off).sum().backward()
    one = torch.ones(x.size(0), w.size(1), device="cuda", dtype=torch.float64)
    assert torch.equal(x.grad.double(), torch.cat([one[a:b] @ w[g].detach().double() for g, (a, b) in enumerate(zip(starts, starts[1:]))]))
    assert torch.equal(w.grad.double(), torch.stack([one[a:b].t() @ x[a:b].detach().double() for a, b in zip(starts, starts[1:])]))


def test_rows_in_no_group_have_no_gradient():
    x, w, off, starts = case(starts=(3, 9, 9, 20))
    x = torch.cat([x, whole(5, x.size(1), seed=7)])
    torch.cuda.empty_cache()
    torch.full((1 << 20,), float("nan"), device="cuda", dtype=torch.bfloat16)  # what an unwritten gradient would hold
    check(x, w, off, starts, whole(x.size(0), w.size(1), seed=3))


@pytest.mark.parametrize("which", ["x", "w"])
def test_only_what_is_asked_for(which, monkeypatch):
    called = []
    for name in ("grouped_gemm_dx", "grouped_gemm_dw"):
        f = getattr(ozk, name)
        monkeypatch.setattr(ozk, name, lambda *a, f=f, name=name, **k: (called.append(name), f(*a, **k))[1])
    x, w, off, _ = case()
    (x if which == "x" else w).requires_grad_()
    ozk.grouped_gemm(x, w, off).float().square().sum().backward()
    assert called == ["grouped_gemm_dx" if which == "x" else "grouped_gemm_dw"]
    assert (x.grad is None) == (which == "w") and (w.grad is None) == (which == "x")


def test_where_no_graph_is_recorded():
    x, w, off, _ = case()
    assert not ozk.grouped_gemm(x, w, off).requires_grad
    w.requires_grad_()
    with torch.no_grad():
        assert not ozk.grouped_gemm(x, w, off).requires_grad
    out = torch.empty(x.size(0), w.size(1), device="cuda", dtype=x.dtype)
    assert not ozk.grouped_gemm(x, w, off, out=out).requires_grad
    assert torch.equal(out, ozk.grouped_gemm(x, w, off).detach())


def test_second_derivatives_are_refused():
    x, w, off, _ = case()
    x.requires_grad_(), w.requires_grad_()
    g, = torch.autograd.grad(ozk.grouped_gemm(x, w, off).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), w)


def test_on_a_stream_of_its_own():
    x, w, off, starts = case()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x, w = x.requires_grad_(), w.requires_grad_()
    y = ozk.grouped_gemm(x, w, off, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y.float().square().sum().backward()
    torch.cuda.synchronize()
    hx, hw = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    h = plain(hx, hw, starts)
    (h * (2 * y.detach().double())).sum().backward()
    assert torch.equal(y.detach().double(), h.detach())
    # 2 y is whole and below 2^9: exact in bf16; the sums of its products are rounded once
    for got, want in ((x.grad, hx.grad), (w.grad, hw.grad)):
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
