"""The operators together, as examples/gated_layer.py uses them: a layer's
result and gradients, and its serving in 4 bits, against 64-bit forms."""
import importlib.util
import os

import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_forward(m, layer, x, w1, w2, rounded=lambda t: t):
    rows, offsets, p = m.route(x, layer.router, layer.top)
    starts, H = offsets.tolist(), w1.shape[1] // 2
    y = []
    for g, (a, b) in enumerate(zip(starts, starts[1:])):
        pre = x[rows[a:b]].double() @ w1[g].t()
        y.append(rounded(torch.nn.functional.silu(pre[:, :H]) * pre[:, H:]) @ w2[g].t())
    return torch.zeros_like(x, dtype=torch.float64).index_add(0, rows, torch.cat(y) * p[:, None].double())


def rows_of(n, width, seed):
    return torch.randn(n, width, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_gradients_of_the_layer(example):
    """h, the slopes and the gradients of the projections are each rounded to bf16 (2^-8 of a value): six roundings on
    the way to a weight's gradient, each of them below 0.4% of the norm."""
    layer = example.GatedLayer(128, 256, experts=5, top=2, seed=3)
    x = rows_of(300, 128, 1)
    r = torch.randn(300, 128, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    (layer.train_forward(x) * r).sum().backward()
    w1, w2 = layer.w1.detach().double().requires_grad_(), layer.w2.detach().double().requires_grad_()
    (plain_forward(example, layer, x, w1, w2) * r.double()).sum().backward()
    for got, want in ((layer.w1.grad, w1.grad), (layer.w2.grad, w2.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 6 * 2.0 ** -8
    assert ozk.ozk_stream_status() == 0


@pytest.mark.parametrize("rows", [1, 4, 40])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_served_rows_are_those_of_the_4_bit_weights(example, rows, fmt):
    """Against the same layer with the values that the 4-bit weights stand for: what is left is h's rounding to bf16."""
    layer = example.GatedLayer(192, 320, experts=6, top=2, seed=4)
    x = rows_of(rows, 192, 5)
    weights = layer.quantize(fmt)
    w1, w2 = ((ozk.mx4_dequantize(q, torch.float64) * scale).view(shape)
              for (q, scale), shape in zip(weights, (layer.w1.shape, layer.w2.shape)))
    got, want = layer.serve(x, weights), plain_forward(example, layer, x, w1, w2)
    assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8
    exact = plain_forward(example, layer, x, w1, w2, rounded=lambda t: t.bfloat16().double())
    assert float((got.double() - exact).norm() / exact.norm()) < 2.0 ** -8
    assert ozk.ozk_stream_status() == 0


def test_a_training_run(example):
    """It runs, and leaves finite weights."""
    layer = example.GatedLayer(64, 96, experts=4, top=2, seed=6)
    x = rows_of(200, 64, 7)
    example.train(layer, x, torch.zeros(200, 64, device="cuda"), 3, rate=1.0)
    assert bool(torch.isfinite(layer.w1).all()) and bool(torch.isfinite(layer.w2).all())
    assert ozk.ozk_stream_status() == 0
