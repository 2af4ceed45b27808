"""The operators together, as examples/expert_layer.py uses them: gradients
through both products against torch's own of the same layer in 64 bits, a
training run, and 4-bit serving."""
import importlib.util
import os

import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_forward(m, layer, x, w1, w2):
    rows, offsets, p = m.route(x, layer.router, layer.top)
    starts = offsets.tolist()
    y = torch.cat([torch.relu(x[rows[a:b]].double() @ w1[g].t()) @ w2[g].t() for g, (a, b) in enumerate(zip(starts, starts[1:]))])
    return torch.zeros_like(x, dtype=torch.float64).index_add(0, rows, y * p[:, None].double())


def test_gradients_of_the_layer(example):
    """bf16 intermediates (2^-9 each way through two products, a relu and the sums' roundings) keep a gradient within 2%."""
    layer = example.ExpertLayer(128, 256, experts=5, top=2, seed=3)
    x = torch.randn(300, 128, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    r = torch.randn(300, 128, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    (layer.train_forward(x) * r).sum().backward()
    w1, w2 = layer.w1.detach().double().requires_grad_(), layer.w2.detach().double().requires_grad_()
    (plain_forward(example, layer, x, w1, w2) * r.double()).sum().backward()
    for got, want in ((layer.w1.grad, w1.grad), (layer.w2.grad, w2.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 0.02


def test_training_lowers_the_loss_and_serving_follows(example):
    teacher = example.ExpertLayer(256, 512, experts=6, top=2, seed=1)
    layer = example.ExpertLayer(256, 512, experts=6, top=2, seed=2)
    layer.router = teacher.router
    x = torch.randn(1024, 256, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()
    with torch.no_grad():
        target = teacher.train_forward(x)
    losses = example.train(layer, x, target, 40, rate=20.0)
    assert losses[-1] < 0.7 * losses[0]
    with torch.no_grad():
        want = layer.train_forward(x)
        for fmt in ("nvfp4", "mxfp4"):
            weights = layer.quantize(fmt)
            got = layer.serve(x, weights)
            # 4-bit rounding of both operands of both products: some tenths of the outputs' size, no more
            assert float((got - want).norm() / want.norm()) < 0.35
            one = layer.serve(x[:1], weights)  # a single row: most experts get none
            assert float((one - got[:1]).norm() / got[:1].norm()) < 0.05
    assert ozk.ozk_stream_status() == 0
