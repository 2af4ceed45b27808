"""What examples/expert_layer.py serves: weights of size 1 / sqrt(width) keep the accuracy that the format has when its
block scales are normal numbers.  By the 64-bit form of tests/lowp_reference.py normal weights then lose 0.095 of their
norm; with block scales among E4M3's subnormals 0.108 at a width of 4096 and 0.120 at 8192."""
import pytest
import torch

from fp64_gemm_emulation_exponent_gb300 import ozk
from test_gpu_expert_layer import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [4096, 8192])
def test_nvfp4_weights_keep_their_accuracy(example, width):  # noqa: F811
    layer = example.ExpertLayer(width, 128, experts=2, top=1, seed=4)
    fmt, (w1, scale1), _ = layer.quantize("nvfp4")
    want = layer.w1.detach().double().view(-1, width)
    got = ozk.mx4_dequantize(w1, torch.float64) * scale1
    assert float((got - want).norm() / want.norm()) < 0.097


def test_served_outputs(example):  # noqa: F811
    """Two quantised operands of independent errors of 0.095, twice: within 0.095 x sqrt(4) = 0.19 of the exact layer's
    outputs, and bf16's own error, with the relu taking some of it."""
    layer = example.ExpertLayer(4096, 512, experts=2, top=1, seed=5)
    x = torch.randn(256, 4096, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    with torch.no_grad():
        want = layer.train_forward(x)
        got = layer.serve(x, layer.quantize("nvfp4"))
    assert float((got - want).norm() / want.norm()) < 0.2


def test_weights_of_one_value(example):  # noqa: F811
    for value in (0.0, 1e-30, 3.0):
        q, scale = example.in_range(torch.full((2, 8, 64), value, device="cuda"), "nvfp4")
        got = ozk.mx4_dequantize(q, torch.float64) * scale
        assert float((got - value).abs().max()) <= 0.07 * value  # E4M3 to 2^-4 of the scale, the code 6 exact
