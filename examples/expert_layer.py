"""A layer of experts trained in bf16 and served in 4 bits, through the
library's grouped and microscaled 4-bit products.

Every row goes to the best experts of a linear router; the rows are sorted by
expert (on the GPU: no count ever reaches the host), and each expert's two
matrices are applied to its own rows:

    h = relu(x W1_e^T)        y = sum over the row's experts of p_e (h W2_e^T)

Training runs ozk.grouped_gemm, whose gradients autograd takes from
ozk.grouped_gemm_dx and ozk.grouped_gemm_dw; serving quantises the weights once (ozk.mx4_quantize) and
each call's rows as they come, and multiplies them with ozk.mx4_grouped_gemm.

    python examples/expert_layer.py [--rows 4096] [--experts 8] [--steps 30]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp64_gemm_emulation_exponent_gb300 import ozk  # noqa: E402


def route(x, router, top):
    """(row of every expert's entry, expert offsets, weight of every entry): entries sorted by expert."""
    weight, expert = torch.topk(torch.softmax(x.float() @ router, dim=1), top, dim=1)
    expert, order = torch.sort(expert.flatten(), stable=True)
    offsets = torch.searchsorted(expert, torch.arange(router.size(1) + 1, device=x.device)).int()
    return order // top, offsets, weight.flatten()[order]


def in_range(w, fmt):
    """w in 4 bits, and the factor that its products take back.  Weights of size 1 / sqrt(width) have block scales among
    E4M3's subnormals, whose few bits cost accuracy (rounding error 0.120 of the weights at a width of 8192, 0.108 at
    4096); a power of two that brings the largest weight to the top of the scales' range, 6 x 448, keeps it at 0.095."""
    top = float(w.abs().max()) if fmt == "nvfp4" else 0.0
    scale = 2.0 ** min(math.floor(math.log2(6 * 448 / top)), 126) if 0.0 < top < math.inf else 1.0
    return ozk.mx4_quantize(w, fmt, prescale=scale), 1.0 / scale


class ExpertLayer:
    def __init__(self, width, hidden, experts, top, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.top = top
        self.router = rand(width, experts) / width ** 0.5
        self.w1 = (rand(experts, hidden, width) / width ** 0.5).bfloat16().requires_grad_()
        self.w2 = (rand(experts, width, hidden) / hidden ** 0.5).bfloat16().requires_grad_()

    def train_forward(self, x):
        rows, offsets, p = route(x, self.router, self.top)
        h = torch.relu(ozk.grouped_gemm(x[rows], self.w1, offsets))
        y = ozk.grouped_gemm(h, self.w2, offsets)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, rows, y.float() * p[:, None])

    def quantize(self, fmt="nvfp4"):
        """The weights in 4 bits, as serving keeps them."""
        return fmt, in_range(self.w1.detach(), fmt), in_range(self.w2.detach(), fmt)

    def serve(self, x, weights):
        fmt, (w1, scale1), (w2, scale2) = weights
        rows, offsets, p = route(x, self.router, self.top)
        h = torch.relu(ozk.mx4_grouped_gemm(ozk.mx4_quantize(x[rows], fmt, offsets=offsets), w1, alpha=scale1))
        y = ozk.mx4_grouped_gemm(ozk.mx4_quantize(h, fmt, offsets=offsets), w2, alpha=scale2)
        return torch.zeros_like(x, dtype=torch.float32).index_add(0, rows, y.float() * p[:, None])


def train(layer, x, target, steps, rate):
    """Plain gradient descent; the loss of every step."""
    losses = []
    for _ in range(steps):
        loss = (layer.train_forward(x) - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for w in (layer.w1, layer.w2):
                w -= rate * w.grad
                w.grad = None
        losses.append(float(loss.detach()))
    return losses


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
    teacher = ExpertLayer(a.width, a.hidden, a.experts, a.top, seed=1)
    layer = ExpertLayer(a.width, a.hidden, a.experts, a.top, seed=2)
    layer.router = teacher.router
    with torch.no_grad():
        target = teacher.train_forward(x)
    losses = train(layer, x, target, a.steps, rate=20.0)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    with torch.no_grad():
        want = layer.train_forward(x)
        for fmt in ("nvfp4", "mxfp4"):
            got = layer.serve(x, layer.quantize(fmt))
            print(f"{fmt}: served outputs within {float((got - want).norm() / want.norm()):.3f} of the bf16 layer's")
    if ozk.ozk_stream_status() != 0:
        raise SystemExit("the device reported a fault")


if __name__ == "__main__":
    main()
