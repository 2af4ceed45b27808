"""16-bit results of a width that is no multiple of 8, as the first columns of wider rows that start on 16 bytes: the
columns beside them belong to the caller and keep what they hold."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu


def whole(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)


def rows_of(t):
    """t with rows 16 bytes apart in multiples."""
    buf = torch.zeros(*t.shape[:-1], -(-t.shape[-1] // 8) * 8, device="cuda", dtype=t.dtype)
    buf[..., : t.shape[-1]] = t
    return buf[..., : t.shape[-1]]


def product(op, cols, dtype):
    """(call with an output, the output's shape, the 64-bit result)"""
    starts = [0, 100, 100, 165]
    spans, off = list(zip(starts, starts[1:])), torch.tensor(starts, dtype=torch.int32, device="cuda")
    T, terms = starts[-1], 72
    if op == "forward":
        x, w = whole(T, terms, seed=1, dtype=dtype), whole(3, cols, terms, seed=2, dtype=dtype)
        return (lambda out: ozk.grouped_gemm(x, w, off, out=out), (T, cols),
                torch.cat([x[a:b].double() @ w[g].double().t() for g, (a, b) in enumerate(spans)]))
    if op == "dx":
        dy, w = whole(T, terms, seed=1, dtype=dtype), rows_of(whole(3, terms, cols, seed=2, dtype=dtype))
        return (lambda out: ozk.grouped_gemm_dx(dy, w, off, out=out), (T, cols),
                torch.cat([dy[a:b].double() @ w[g].double() for g, (a, b) in enumerate(spans)]))
    if op == "dw":
        dy, x = whole(T, terms, seed=1, dtype=dtype), rows_of(whole(T, cols, seed=2, dtype=dtype))
        return (lambda out: ozk.grouped_gemm_dw(dy, x, off, out=out), (3, terms, cols),
                torch.stack([dy[a:b].double().t() @ x[a:b].double() for a, b in spans]))
    a, b = whole(T, terms, seed=1).float(), whole(3 * cols, terms, seed=2).float()
    a[:, ::16], b[:, ::16] = 6.0, -6.0  # every block's scale 1
    w = b.view(3, cols, terms)
    qa, qw = ozk.mx4_quantize(a, op, offsets=off), ozk.mx4_quantize(w, op)
    return (lambda out: ozk.mx4_grouped_gemm(qa, qw, out=out), (T, cols),
            torch.cat([a[s:e].double() @ w[g].double().t() for g, (s, e) in enumerate(spans)]))


@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("op", ["forward", "dx", "dw", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("cols,pad", [(5, 3), (61, 3), (63, 1), (66, 14), (77, 11), (130, 6), (191, 65), (250, 6), (313, 7)])
def test_columns_beside_a_result_are_kept(cols, pad, op, dtype, pairs):
    call, shape, want = product(op, cols, dtype)
    buf = torch.full((*shape[:-1], cols + pad), 9.0, device="cuda", dtype=dtype)
    assert (cols + pad) % 8 == 0 and buf.data_ptr() % 16 == 0
    if hasattr(ozk, "ozk_withhold_next_product"):
        ozk.ozk_withhold_next_product(pairs, 0, -1, 1000000)  # this tile form
    call(buf[..., :cols])
    assert torch.equal(buf[..., :cols], want.to(dtype))
    assert bool((buf[..., cols:] == 9).all())
    assert ozk.ozk_stream_status() == 0
