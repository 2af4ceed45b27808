"""A gated feed-forward layer of experts, trained in bf16 and served token by
token with 4-bit weights.

Every row goes to the best experts of a linear router, is sorted by expert (on
the GPU), and each expert applies its three matrices to its own rows:

    h = silu(x Wg_e^T) * (x Wu_e^T)        y = sum over the row's experts of p_e (h W_e^T)

Training runs ozk.grouped_gated_gemm (both projections, the activation and the
product in one kernel) and ozk.grouped_gemm, whose gradients autograd takes
from the library; serving quantises the weights once and runs a few rows at a
time through ozk.mx4_gated_gemv and ozk.mx4_gemv, the rows in 16 bits.

    python examples/gated_layer.py [--rows 4096] [--experts 8] [--steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from expert_layer import in_range, route, train  # noqa: E402
from fp64_gemm_emulation_exponent_gb300 import ozk  # noqa: E402


class GatedLayer:
    def __init__(self, width, hidden, experts, top, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.top = top
        self.router = rand(width, experts) / width ** 0.5
        self.w1 = (rand(experts, 2 * hidden, width) / width ** 0.5).bfloat16().requires_grad_()  # the gate's rows first
        self.w2 = (rand(experts, width, hidden) / hidden ** 0.5).bfloat16().requires_grad_()

    def train_forward(self, x):
        rows, offsets, p = route(x, self.router, self.top)
        h = ozk.grouped_gated_gemm(x[rows], self.w1, offsets)
        y = ozk.grouped_gemm(h, self.w2, offsets)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, rows, y.float() * p[:, None])

    def quantize(self, fmt="nvfp4"):
        """The weights in 4 bits, as serving keeps them."""
        return in_range(self.w1.detach(), fmt), in_range(self.w2.detach(), fmt)

    def serve(self, x, weights):
        (w1, scale1), (w2, scale2) = weights
        rows, offsets, p = route(x, self.router, self.top)
        h = ozk.mx4_gated_gemv(x[rows], w1, offsets, alpha=scale1)
        y = ozk.mx4_gemv(h, w2, offsets, alpha=scale2, out_dtype=torch.float32)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, rows, y * p[:, None])


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--rows", type=int, default=4096)
    a.add_argument("--width", type=int, default=1024)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--experts", type=int, default=8)
    a.add_argument("--top", type=int, default=2)
    a.add_argument("--steps", type=int, default=30)
    a = a.parse_args()
    x = torch.randn(a.rows, a.width, device="cuda").bfloat16()
    teacher = GatedLayer(a.width, a.hidden, a.experts, a.top, seed=1)
    layer = GatedLayer(a.width, a.hidden, a.experts, a.top, seed=2)
    layer.router = teacher.router
    with torch.no_grad():
        target = teacher.train_forward(x)
    losses = train(layer, x, target, a.steps, rate=20.0)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    with torch.no_grad():
        few = x[:4]
        want = layer.train_forward(few)
        for fmt in ("nvfp4", "mxfp4"):
            got = layer.serve(few, layer.quantize(fmt))
            print(f"{fmt}: served outputs within {float((got - want).norm() / want.norm()):.3f} of the bf16 layer's")
    if ozk.ozk_stream_status() != 0:
        raise SystemExit("the device reported a fault")


if __name__ == "__main__":
    main()
