"""Large 4-bit matrices bit for bit: from about 14000 chunks of 512 columns on a warp quantises (and dequantises) a run
of two to four chunks of a row, the next one loading while it works on one, and the last run of a row may be shorter."""
import numpy as np
import pytest
import torch

import lowp_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
WARPS = 48  # an SM has so many before runs get longer
# rows, columns: runs of 2 and 3 in 9 chunks, of 2 and 4 in 5, of 2 in 16 (148 or 152 SMs)
SIZES = [(2000, 4500), (2700, 4500), (3400, 2090), (14000, 2090), (1100, 8192)]


def run_length(rows, K, fmt):
    span = 128 if fmt == "mxfp4" else 64
    columns = -(-ref.kpad(K) // span) * span
    chunks = -(-columns // 512)
    sms = ozk.lib().ozk_device_sm_count()
    return min(4, chunks, max(rows * chunks // (sms * WARPS), 1)), chunks


def stored_scales(scales, rows, K, fmt):
    """Scale bytes [rows, blocks] of a matrix of one group."""
    blocks = ref.kpad(K) // ref.BLOCK[fmt]
    tiles = -(-blocks // 4)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    return scales[(r // 128 * tiles + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4]


def spread(rows, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g, device="cuda")
    e = torch.randint(-6, 7, (rows, -(-K // 16)), generator=g, device="cuda").repeat_interleave(16, dim=1)[:, :K]
    return torch.ldexp(x, e).to(dtype)


def view(rows, K, align, dtype, fill):
    """[rows, K] whose rows start on `align` bytes and, of the next power of two, not all."""
    size = torch.empty(0, dtype=dtype).element_size()
    step = align // size  # elements
    ld = -(-K // step) * step
    if align < 32 and ld // step % 2 == 0:
        ld += step
    buf = torch.full((rows * ld + 64,), fill, device="cuda", dtype=dtype)
    start = step if align < 32 else 0
    return buf, buf[start: start + rows * ld].view(rows, ld)[:, :K]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("dtype,align", [(torch.bfloat16, 32), (torch.bfloat16, 16), (torch.float16, 4), (torch.bfloat16, 2),
                                         (torch.float32, 32), (torch.float32, 4)])
def test_runs_of_chunks_bit_exact(fmt, rows, K, dtype, align):
    run, chunks = run_length(rows, K, fmt)
    assert run > 1
    values = spread(rows, K, dtype)
    _, x = view(rows, K, align, dtype, float("nan"))
    x.copy_(values)
    q = ozk.mx4_quantize(x, fmt)
    code, neg, byte = ref.quantize(values.double().cpu().numpy(), fmt)
    got_code, got_neg = ref.stored_codes(q.codes.cpu().numpy(), K)
    assert np.array_equal(stored_scales(q.scales.cpu().numpy(), rows, K, fmt), byte)
    assert np.array_equal(got_code, code)
    assert np.array_equal(got_neg & (got_code > 0), neg & (code > 0))
    buf, out = view(rows, K, align, dtype, 7.0)
    ozk.mx4_dequantize(q, out=out)
    want = torch.from_numpy(ref.values(code, neg, byte, fmt, K)).to(dtype)  # a product of few bits: exact
    assert torch.equal(out.cpu(), want)
    out.fill_(7.0)
    assert bool((buf == 7.0).all())
    assert ozk.ozk_stream_status() == 0


def test_the_sizes_cover_every_run():
    lengths = [run_length(*size, fmt) for size in SIZES for fmt in ("nvfp4", "mxfp4")]
    assert {run for run, _ in lengths} == {2, 3, 4}
    assert any(chunks % run for run, chunks in lengths) and any(chunks % run == 0 for run, chunks in lengths)
