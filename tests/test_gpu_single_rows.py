"""Grouped products whose operands are one row (a single token, weights of one
output): views of padded buffers give the results that two rows of the same
buffers give, the columns beside them having no part in them."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk


def padded(*shape, cols, seed, device="cuda", fill=float("nan")):
    """Small whole numbers [*shape, cols] in a buffer of 64 columns, `fill` beside them."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((*shape, 64), fill)
    buf[..., :cols] = torch.randint(-2, 3, (*shape, cols), generator=g).float()
    return buf.bfloat16().to(device)[..., :cols]


@pytest.mark.parametrize("cols", [1, 7, 8, 60, 64])
def test_leading_dimension_of_one_row(cols):
    """With one row nothing is addressed by it; what is passed has to suit a bulk copy all the same."""
    t = padded(4, cols=cols, seed=1, device="cpu")
    assert ozk._rows(t[:2])[2] == 64
    for one in (t[:1], t[:1].contiguous(), t[0].unsqueeze(0), t[:1].expand(1, cols)):
        rows, c, ld = ozk._rows(one)
        assert (rows, c) == (1, cols) and ld >= cols and ld % 8 == 0
    w = padded(3, 2, cols=cols, seed=2, device="cpu")
    assert ozk._groups(w)[3:] == (64, 128)
    g, r, c, ld, stride = ozk._groups(w[:, :1])
    assert (g, r, c, stride) == (3, 1, cols, 128) and ld >= cols and ld % 8 == 0
    assert ozk._groups(w[:1, :1])[3] % 8 == 0



@pytest.mark.gpu
@pytest.mark.parametrize("cols", [8, 60])
@pytest.mark.parametrize("rows", [1, 2])
def test_products_of_a_single_token(rows, cols):
    """T = 1 with K, N = cols and 24 on buffers padded to 64 columns."""
    G, N = 3, 24
    off = torch.tensor([0, 0, rows, rows], dtype=torch.int32, device="cuda")
    x, w = padded(4, cols=cols, seed=1)[:rows], padded(G, N, cols=cols, seed=2)
    y = ozk.grouped_gemm(x, w, off)
    assert torch.equal(y.double(), x.double() @ w[1].double().t())
    dy, v = padded(4, cols=cols, seed=3)[:rows], padded(G, cols, cols=N, seed=4)
    assert torch.equal(ozk.grouped_gemm_dx(dy, v, off).double(), dy.double() @ v[1].double())
    dw = ozk.grouped_gemm_dw(dy, x, off)
    assert torch.equal(dw[1].double(), dy.double().t() @ x.double()) and bool((dw[[0, 2]] == 0).all())
    out = torch.full((2, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    ozk.grouped_gemm_dx(dy, padded(G, cols, cols=cols, seed=5), off, out=out[:rows, :cols])
    assert bool((out[:, cols:] == 9).all()) and bool((out[rows:] == 9).all())
    assert ozk.ozk_stream_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [8, 60])
@pytest.mark.parametrize("G", [1, 3])
def test_products_with_one_output(G, cols):
    """N = 1: one row of weights a group, 64 columns apart."""
    starts = [0, 7] if G == 1 else [0, 3, 3, 7]
    off = torch.tensor(starts, dtype=torch.int32, device="cuda")
    x, w = padded(7, cols=cols, seed=1), padded(G, 1, cols=cols, seed=2)
    dy = padded(7, cols=1, seed=3)
    spans = list(zip(starts, starts[1:]))
    assert torch.equal(ozk.grouped_gemm(x, w, off).double(),
                       torch.cat([x[a:b].double() @ w[g].double().t() for g, (a, b) in enumerate(spans)]))
    assert torch.equal(ozk.grouped_gemm_dx(dy, w, off).double(),
                       torch.cat([dy[a:b].double() @ w[g].double() for g, (a, b) in enumerate(spans)]))
    out = torch.full((G, 1, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    ozk.grouped_gemm_dw(dy, x, off, out=out[..., :cols])
    assert torch.equal(out[..., :cols].double(), torch.stack([dy[a:b].double().t() @ x[a:b].double() for a, b in spans]))
    assert bool((out[..., cols:] == 9).all())
    assert ozk.ozk_stream_status() == 0
