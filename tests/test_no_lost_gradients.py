"""Calls that record no gradient, or no forward-mode tangent, say so instead of
dropping it (the host side, with the stand-ins of test_operand_device)."""
import pytest
import torch
from torch.autograd import forward_ad

from fp64_gemm_emulation_exponent_gb300 import ozk
from test_operand_device import FakeTensor, machine, matrix, offsets, tensor  # noqa: F401


def asking(*shape):
    t = tensor(*shape)
    t.requires_grad = True
    return t


ROWS = {
    "mx4_gemv": lambda x, **k: ozk.mx4_gemv(x, matrix(groups=2), offsets(), **k),
    "mx4_gated_gemv": lambda x, **k: ozk.mx4_gated_gemv(x, matrix(), **k),
}


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("device", [0, 1])
def test_rows_that_ask_for_a_gradient(machine, name, device):  # noqa: F811
    machine.fake.current = device  # the rows' own device, or another one
    with pytest.raises(NotImplementedError, match="gradient"):
        ROWS[name](asking(4, 64))
    assert machine.calls == [] and machine.fake.allocated_on == []
    ROWS[name](asking(4, 64), out=tensor(4, 8))  # into memory given
    machine.fake.is_grad_enabled = lambda: False
    ROWS[name](asking(4, 64))
    assert [c[0] for c in machine.calls] == ["ozk_" + name] * 2


CALLS = {
    "grouped_gemm, rows": lambda d: ozk.grouped_gemm(d((16, 64)), tensor(2, 32, 64), offsets()),
    "grouped_gemm, weights": lambda d: ozk.grouped_gemm(tensor(16, 64), d((2, 32, 64)), offsets()),
    "grouped_gated_gemm, rows": lambda d: ozk.grouped_gated_gemm(d((16, 64)), tensor(2, 64, 64), offsets()),
    "grouped_gated_gemm, weights": lambda d: ozk.grouped_gated_gemm(tensor(16, 64), d((2, 64, 64)), offsets()),
    "mx4_gemv": lambda d: ozk.mx4_gemv(d((4, 64)), matrix(groups=2), offsets()),
    "mx4_gated_gemv": lambda d: ozk.mx4_gated_gemv(d((4, 64)), matrix()),
}


@pytest.mark.parametrize("name", CALLS)
def test_tangents(machine, monkeypatch, name):  # noqa: F811
    """A tangent is refused, with gradients off too: no_grad is not meant for forward mode."""
    class Dual(FakeTensor):
        tangent = True

    monkeypatch.setattr(ozk, "_forward_ad", forward_ad)
    monkeypatch.setattr(forward_ad, "unpack_dual", lambda t: (t, getattr(t, "tangent", None)))
    dual = lambda shape: Dual(shape, torch.bfloat16, 1)  # noqa: E731
    plain = lambda shape: tensor(*shape)  # noqa: E731
    machine.fake.is_grad_enabled = lambda: False
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError, match="tangent"):
            CALLS[name](dual)
        assert machine.calls == []
        CALLS[name](plain)
    CALLS[name](plain)
    assert len(machine.calls) == 2


def test_what_counts_as_a_tangent(monkeypatch):
    monkeypatch.setattr(ozk, "_forward_ad", forward_ad)

    def refused(*tensors):
        try:
            ozk._no_tangents("a call", *tensors)
        except NotImplementedError:
            return True
        return False

    x = torch.ones(3)
    assert not refused(x)
    with forward_ad.dual_level():
        assert not refused(x, x)
        d = forward_ad.make_dual(x, x)
        assert refused(d) and refused(x, d)
        with torch.no_grad():
            assert refused(d)
        assert not refused(forward_ad.unpack_dual(d).primal)
    assert not refused(x)


def test_a_function_with_a_derivative_of_its_own_may_call_them(monkeypatch):
    """Inside a custom function's forward there are no tangents, and no gradients are recorded."""
    monkeypatch.setattr(ozk, "_forward_ad", forward_ad)

    class Double(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            ozk._no_tangents("a call", x)
            assert not torch.is_grad_enabled()
            return 2 * x

        @staticmethod
        def jvp(ctx, tangent):
            return 2 * tangent

    x = torch.ones(3)
    with forward_ad.dual_level():
        assert torch.equal(forward_ad.unpack_dual(Double.apply(forward_ad.make_dual(x, x))).tangent, 2 * x)


@pytest.mark.gpu
def test_on_the_gpu():
    """The same calls on real tensors."""
    x, w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 32, 64, dtype=torch.bfloat16, device="cuda")
    at, q = torch.tensor([0, 4], dtype=torch.int32, device="cuda"), ozk.mx4_quantize(w)
    calls = [lambda x: ozk.grouped_gemm(x, w, at), lambda x: ozk.grouped_gated_gemm(x, w, at), lambda x: ozk.mx4_gemv(x, q),
             lambda x: ozk.mx4_gated_gemv(x, q)]
    wanted = [call(x) for call in calls]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call, want in zip(calls, wanted):
            with pytest.raises(NotImplementedError):
                call(dual)
            assert torch.equal(call(x), want)
            assert torch.equal(call(forward_ad.unpack_dual(dual).primal), want)
    asking = x.clone().requires_grad_()
    for call, want in zip(calls[:2], wanted):
        assert call(asking).requires_grad
    for call, want in zip(calls[2:], wanted[2:]):
        with pytest.raises(NotImplementedError):
            call(asking)
        with torch.no_grad():
            assert torch.equal(call(asking), want)
    assert torch.equal(ozk.mx4_gemv(asking, q, out=torch.empty_like(wanted[2])), wanted[2])
    assert ozk.ozk_stream_status() == 0
