"""Calls run on the device that holds their operands, whichever is current: the
host side, with stand-ins for torch, its tensors and the library that record
which device was current at each launch and whose stream it was given."""
import contextlib
import math

import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk


class FakeTensor:
    def __init__(self, shape, dtype, index, storage=1 << 40):
        self.shape, self.dtype, self.index, self.storage = tuple(shape), dtype, index, storage
        self.device = f"cuda:{index}"
        self.requires_grad = False

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.storage

    def stride(self, dim=None):
        s = tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))
        return s if dim is None else s[dim]

    def size(self, dim):
        return self.shape[dim]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True

    def view(self, *shape):
        return FakeTensor(shape, self.dtype, self.index)


class FakeStream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 0x5000 + index


class FakeTorch:
    """A machine of several devices; the first is current."""

    def __init__(self):
        self.current = 0
        self.on, self.allocated_on = None, []
        for name in ("int32", "uint8", "bfloat16", "float16", "float32", "float64"):
            setattr(self, name, getattr(torch, name))
        self._C = self.cuda = self

    def _cuda_getDevice(self):
        return self.current

    current_device = _cuda_getDevice

    def _cuda_getCurrentRawStream(self, index):
        return 0x1000 + index

    @contextlib.contextmanager
    def device(self, index):
        before, self.current = self.current, self.current if index is None else index
        try:
            yield
        finally:
            self.current = before

    @contextlib.contextmanager
    def stream(self, s):
        before, self.on = self.on, s or self.on
        with self.device(self.current if s is None else s.device_index):
            yield
        self.on = before

    def is_grad_enabled(self):
        return True

    def empty(self, *shape, dtype=None, device=None):
        shape = shape[0] if isinstance(shape[0], tuple) else shape
        self.allocated_on.append(self.on)
        return FakeTensor(shape, dtype, int(str(device)[5:]), storage=1 << 42)


class FakeLibrary:
    """Every entry point succeeds and notes (name, device current, stream handle)."""

    def __init__(self, fake):
        self.fake, self.calls = fake, []

    def __getattr__(self, name):
        def entry(*args):
            values = [getattr(a, "value", a) for a in args]
            streams = [v for v in values if isinstance(v, int) and (0x1000 <= v < 0x1010 or 0x5000 <= v < 0x5010)]
            self.calls.append((name, self.fake.current, streams[-1]))
            return 0
        return entry


@pytest.fixture
def machine(monkeypatch):
    fake = FakeTorch()
    library = FakeLibrary(fake)
    monkeypatch.setattr(ozk, "_torch", fake)
    monkeypatch.setattr(ozk, "_current_device", fake._cuda_getDevice)
    monkeypatch.setattr(ozk, "_current_stream", fake._cuda_getCurrentRawStream)
    monkeypatch.setattr(ozk, "_lib", library)
    monkeypatch.setattr(ozk, "_DTYPES", {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float64: 3})
    return library


def tensor(*shape, dtype=torch.bfloat16, index=1):
    return FakeTensor(shape, dtype, index)


def matrix(rows=16, K=64, index=1, groups=1, offsets=None):
    codes = tensor(rows, -(-K // 64) * 32, dtype=torch.uint8, index=index)
    scales = tensor(ozk.mx4_scale_bytes(rows, K, "nvfp4", 16), dtype=torch.uint8, index=index)
    return ozk.Mx4(codes, scales, rows, K, "nvfp4", groups, offsets)


def offsets(index=1):
    return tensor(3, dtype=torch.int32, index=index)


LOWP = {
    "ozk_mx4_quantize": lambda i, s: ozk.mx4_quantize(tensor(16, 64, index=i), stream=s),
    "ozk_mx4_dequantize": lambda i, s: ozk.mx4_dequantize(matrix(index=i), torch.float32, stream=s),
    "ozk_mx4_gemm": lambda i, s: ozk.mx4_gemm(matrix(index=i), matrix(index=i), out_dtype=torch.float32, stream=s),
    "ozk_mx4_grouped_gemm": lambda i, s: ozk.mx4_grouped_gemm(
        matrix(index=i, offsets=offsets(i)), matrix(index=i, groups=2), out_dtype=torch.float32, stream=s),
    "ozk_grouped_gemm": lambda i, s: ozk.grouped_gemm(
        tensor(16, 64, index=i), tensor(2, 32, 64, index=i), offsets(i), stream=s),
    "ozk_grouped_gemm_dx": lambda i, s: ozk.grouped_gemm_dx(
        tensor(16, 32, index=i), tensor(2, 32, 64, index=i), offsets(i), stream=s),
    "ozk_grouped_gemm_dw": lambda i, s: ozk.grouped_gemm_dw(
        tensor(16, 32, index=i), tensor(16, 64, index=i), offsets(i), stream=s),
}


@pytest.mark.parametrize("name", LOWP)
@pytest.mark.parametrize("index", [0, 1, 3])
def test_low_precision_calls_run_on_their_operands_device(machine, name, index):
    LOWP[name](index, None)
    LOWP[name](index, FakeStream(index))
    assert machine.calls == [(name, index, 0x1000 + index), (name, index, 0x5000 + index)]
    assert machine.fake.current == 0  # left as it was


@pytest.mark.parametrize("name", LOWP)
def test_low_precision_calls_refuse_another_devices_stream(machine, name):
    with pytest.raises(ValueError):
        LOWP[name](1, FakeStream(0))
    assert machine.calls == []


FP64 = {
    "ozk_dgemm": lambda i, s: ozk.dgemm(wide(8, 16, i), wide(16, 4, i), 14, stream=s),
    "ozk_dgemm_norm": lambda i, s: ozk.dgemm(wide(8, 16, i), wide(16, 4, i), 13, scaling="norm", stream=s),
    "ozk_dgemm_bits": lambda i, s: ozk.dgemm(wide(8, 16, i), wide(16, 4, i), target_bits=40, stream=s),
    "ozk_dgemm_ws_timed": lambda i, s: ozk.ozk_dgemm_ws_timed(
        8, 4, 16, wide(8, 16, i), 16, wide(16, 4, i), 4, wide(8, 4, i), 4, 14, wide(1, 1, i), 8, None, stream=s),
    "ozk_quantize_a": lambda i, s: ozk.ozk_quantize_a(8, 16, wide(8, 16, i), 16, wide(8, 1, i), 14, wide(8, 64, i), stream=s),
}


def wide(rows, cols, index):
    return tensor(rows, cols, dtype=torch.float64, index=index)


@pytest.mark.parametrize("name", FP64)
@pytest.mark.parametrize("index", [0, 2])
def test_fp64_calls_run_on_their_operands_device(machine, name, index):
    FP64[name](index, None)
    FP64[name](index, FakeStream(index))
    assert machine.calls == [(name, index, 0x1000 + index), (name, index, 0x5000 + index)]
    with pytest.raises(ValueError):
        FP64[name](index, FakeStream(index + 1))
    with pytest.raises(ValueError):
        ozk.dgemm(wide(8, 16, index), wide(16, 4, index + 1), 14)
    assert machine.fake.current == 0 and len(machine.calls) == 2


def test_host_operands_run_on_the_streams_device(machine):
    host = [wide(8, 8, -1) for _ in range(3)]
    ozk.ozk_dgemm_host(8, 8, 8, host[0], 8, host[1], 8, host[2], 8, 14)
    ozk.ozk_dgemm_host_async(8, 8, 8, host[0], 8, host[1], 8, host[2], 8, 14, stream=FakeStream(2))
    assert machine.calls == [("ozk_dgemm_host", 0, 0x1000), ("ozk_dgemm_host_async", 2, 0x5002)]


def test_status_is_that_of_the_streams_device(machine):
    ozk.ozk_stream_status(FakeStream(3))
    assert machine.calls == [("ozk_stream_status", 3, 0x5003)]


RESULTS = {
    "mx4_dequantize": lambda dtype: ozk.mx4_dequantize(matrix(), dtype),
    "mx4_gemm": lambda dtype: ozk.mx4_gemm(matrix(), matrix(), out_dtype=dtype),
    "mx4_grouped_gemm": lambda dtype: ozk.mx4_grouped_gemm(matrix(offsets=offsets()), matrix(groups=2), out_dtype=dtype),
    "grouped_gemm": lambda dtype: ozk.grouped_gemm(tensor(16, 64), tensor(2, 32, 64), offsets(), out_dtype=dtype),
    "grouped_gemm_dx": lambda dtype: ozk.grouped_gemm_dx(tensor(16, 32), tensor(2, 32, 64), offsets(), out_dtype=dtype),
    "grouped_gemm_dw": lambda dtype: ozk.grouped_gemm_dw(tensor(16, 32), tensor(16, 64), offsets(), out_dtype=dtype),
}


@pytest.mark.parametrize("name", RESULTS)
def test_result_types_that_the_library_lacks(machine, name):
    """A TypeError that names the type, before anything is allocated or launched."""
    for dtype in (torch.int32, torch.bool, torch.complex64):
        with pytest.raises(TypeError, match="ozk_dtype"):
            RESULTS[name](dtype)
    assert machine.calls == []


@pytest.mark.parametrize("name", list(LOWP) + ["ozk_dgemm", "ozk_dgemm_norm", "ozk_dgemm_bits"])
def test_results_are_allocated_on_the_stream_that_writes_them(machine, name):
    """Memory that another stream's kernels may still be using must not be handed to it."""
    s = FakeStream(1)
    {**LOWP, **FP64}[name](1, s)
    assert machine.fake.allocated_on == [s]
