"""The gated products' host side, without a GPU: refusals of the entry points
before anything is launched, and the device, stream and allocations of the calls
(with the stand-ins of test_operand_device)."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import build as ozk_build
from fp64_gemm_emulation_exponent_gb300 import ozk
from test_operand_device import FakeStream, machine, matrix, offsets, tensor  # noqa: F401

BIG = 1 << 44  # addresses that nothing dereferences, far apart
X, W, Y, S, P, DH, DX, DW, OFF = (BIG * i for i in range(1, 10))
INVALID, UNSUPPORTED = ozk.OZK_ERR_INVALID_ARG, ozk.OZK_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ozk_build.build()
    yield


def forward(T=4, N=8, K=64, groups=2, off=OFF, x=X, ldx=None, w=W, ldw=None, stride=None, dtype=0, act=0, y=Y, ldy=None, s=S,
            lds=None, plane=None):
    ldw, lds = K if ldw is None else ldw, N if lds is None else lds
    return ozk.lib().ozk_grouped_gated_gemm(T, N, K, groups, off, x, K if ldx is None else ldx, w, ldw,
                                            2 * N * ldw if stride is None else stride, dtype, act, y, N if ldy is None else ldy,
                                            s, lds, T * lds if plane is None else plane, None)


def grad(T=4, N=8, groups=2, off=OFF, dh=DH, lddh=None, s=S, lds=None, plane=None, dtype=0, p=P, ldp=None):
    lds = N if lds is None else lds
    return ozk.lib().ozk_gated_grad(T, N, groups, off, dh, N if lddh is None else lddh, s, lds,
                                    T * lds if plane is None else plane, dtype, p, 2 * N if ldp is None else ldp, None)


def backward(T=4, N=8, K=64, groups=2, off=OFF, dh=DH, lddh=None, s=S, lds=None, plane=None, x=X, ldx=None, w=W, ldw=None,
             stride=None, dtype=0, p=P, ldp=None, dx=DX, lddx=None, dw=DW, lddw=None, dwstride=None):
    lds, ldw, lddw = N if lds is None else lds, K if ldw is None else ldw, K if lddw is None else lddw
    return ozk.lib().ozk_grouped_gated_gemm_grad(
        T, N, K, groups, off, dh, N if lddh is None else lddh, s, lds, T * lds if plane is None else plane, x,
        K if ldx is None else ldx, w, ldw, 2 * N * ldw if stride is None else stride, dtype, p, 2 * N if ldp is None else ldp,
        dx, K if lddx is None else lddx, dw, lddw, 2 * N * lddw if dwstride is None else dwstride, None)


def test_forward_refusals():
    for bad in (dict(T=-1), dict(N=-1), dict(K=-1), dict(groups=0), dict(off=None), dict(act=-1), dict(act=3), dict(x=None),
                dict(w=None), dict(y=None), dict(y=Y + 1), dict(ldx=56), dict(ldw=56), dict(ldy=7), dict(stride=15 * 64),
                dict(s=S + 2), dict(lds=7), dict(plane=31), dict(y=X), dict(y=W), dict(y=S), dict(s=X), dict(s=W)):
        assert forward(**bad) == INVALID, bad
    for bad in (dict(dtype=2), dict(T=1 << 31), dict(N=(1 << 21) + 1), dict(K=(1 << 22) + 1), dict(groups=1025), dict(ldx=68),
                dict(ldw=68), dict(x=X + 8), dict(w=W + 2), dict(stride=16 * 64 + 4)):
        assert forward(**bad) == UNSUPPORTED, bad
    for empty in (dict(T=0), dict(N=0)):
        assert forward(**empty) == ozk.OZK_OK


def test_gradient_refusals():
    for bad in (dict(T=-1), dict(N=-1), dict(groups=0), dict(off=None), dict(dh=None), dict(dh=DH + 1), dict(s=None),
                dict(s=S + 2), dict(p=None), dict(p=P + 1), dict(lddh=7), dict(lds=7), dict(plane=31), dict(ldp=15),
                dict(p=DH), dict(p=S)):
        assert grad(**bad) == INVALID, bad
    for bad in (dict(dtype=2), dict(T=1 << 31), dict(N=(1 << 21) + 1), dict(groups=1025)):
        assert grad(**bad) == UNSUPPORTED, bad
    for empty in (dict(T=0), dict(N=0)):
        assert grad(**empty) == ozk.OZK_OK


def test_backward_refusals():
    for bad in (dict(T=-1), dict(N=-1), dict(K=-1), dict(groups=0), dict(off=None), dict(dh=None), dict(s=None), dict(p=None),
                dict(lddh=7), dict(lds=7), dict(plane=31), dict(ldp=15), dict(x=None), dict(w=None), dict(ldx=56), dict(ldw=56),
                dict(lddx=63), dict(lddw=63), dict(dwstride=15 * 64), dict(dx=DX + 1), dict(p=DH), dict(p=S), dict(p=X), dict(p=W),
                dict(dx=DH), dict(dx=S), dict(dx=X), dict(dx=W), dict(dx=P), dict(dw=DH), dict(dw=S), dict(dw=X), dict(dw=W),
                dict(dw=P), dict(dw=DX)):
        assert backward(**bad) == INVALID, bad
    for bad in (dict(dtype=2), dict(T=1 << 31), dict(N=(1 << 21) + 1), dict(K=(1 << 22) + 1), dict(groups=1025), dict(ldx=68),
                dict(ldw=68), dict(ldp=20), dict(p=P + 8), dict(x=X + 8), dict(w=W + 2)):
        assert backward(**bad) == UNSUPPORTED, bad


def slopes(i):
    return tensor(2, 16, 32, dtype=torch.float32, index=i)


CALLS = {
    "ozk_grouped_gated_gemm": lambda i, s: ozk.grouped_gated_gemm(
        tensor(16, 64, index=i), tensor(2, 64, 64, index=i), offsets(i), stream=s),
    "ozk_gated_grad": lambda i, s: ozk.gated_grad(tensor(16, 32, index=i), slopes(i), offsets(i), stream=s),
    "ozk_grouped_gated_gemm_grad": lambda i, s: ozk.grouped_gated_gemm_grad(
        tensor(16, 32, index=i), tensor(16, 64, index=i), tensor(2, 64, 64, index=i), offsets(i), slopes(i), stream=s),
    "ozk_mx4_gemv": lambda i, s: ozk.mx4_gemv(tensor(4, 64, index=i), matrix(index=i, groups=2), offsets(i), stream=s),
    "ozk_mx4_gated_gemv": lambda i, s: ozk.mx4_gated_gemv(tensor(4, 64, index=i), matrix(index=i), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("index", [0, 1, 3])
def test_calls_run_on_their_operands_device(machine, name, index):  # noqa: F811
    CALLS[name](index, None)
    CALLS[name](index, FakeStream(index))
    assert machine.calls == [(name, index, 0x1000 + index), (name, index, 0x5000 + index)]
    assert machine.fake.current == 0  # left as it was


@pytest.mark.parametrize("name", CALLS)
def test_calls_refuse_another_devices_stream(machine, name):  # noqa: F811
    with pytest.raises(ValueError):
        CALLS[name](1, FakeStream(0))
    assert machine.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_results_are_allocated_on_the_stream_that_writes_them(machine, name):  # noqa: F811
    s = FakeStream(1)
    CALLS[name](1, s)
    assert machine.fake.allocated_on and set(machine.fake.allocated_on) == {s}


def test_operands_of_two_devices(machine):  # noqa: F811
    for call in (lambda: ozk.mx4_gemv(tensor(4, 64, index=0), matrix(index=1)),
                 lambda: ozk.mx4_gemv(tensor(4, 64, index=1), matrix(index=1, groups=2), offsets(0)),
                 lambda: ozk.gated_grad(tensor(16, 32, index=0), slopes(1)),
                 lambda: ozk.grouped_gated_gemm(tensor(16, 64, index=1), tensor(2, 64, 64, index=0), offsets(1)),
                 lambda: ozk.grouped_gated_gemm_grad(tensor(16, 32, index=0), tensor(16, 64, index=1), tensor(2, 64, 64, index=1),
                                                     offsets(1), slopes(1))):
        with pytest.raises(ValueError):
            call()
    assert machine.calls == []
