"""The activations far to the left, where their distribution P is tiny: values
that fp32 holds are not lost, whatever multiplies them; and how exact they are
in the products of a few rows.

P = e^z / (1 + e^z) or a polynomial times e^(-g^2/2) is off by off(z) units of
gated_reference, and by at most 3 of fp32's least steps 2^-149 where e^z is
below 2^-126 (its rounding, and those of two factors below 1): times |g| <= 104
that is below 2^-140, and times |g| z' <= 11 * 17 of the slope, 2^-139."""
import math

import numpy as np
import pytest
import torch

import gated_reference as ref
from fp64_gemm_emulation_exponent_gb300 import ozk

pytestmark = pytest.mark.gpu
SPAN = {"silu": (-104.0, -60.0), "gelu": (-14.0, -9.0), "gelu_tanh": (-11.0, -7.0)}
C = math.sqrt(8 / math.pi)


def exact(g, name):
    """(act(g), the two terms of act'(g) = P + g P') in 64 bits, digits kept in the tails."""
    if name == "gelu":
        p = np.array([math.erfc(-v * math.sqrt(0.5)) / 2 for v in g])
        return g * p, p, g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    z, dz = (g, 1.0) if name == "silu" else (C * (g + 0.044715 * g ** 3), C * (1 + 0.134145 * g * g))
    e = np.exp(-np.abs(z))
    p = np.where(z >= 0, 1, e) / (1 + e)
    return g * p, p, g * (e / (1 + e) ** 2) * dz


def bf16_between(lo, hi):
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    return v[(v >= lo) & (v <= hi)]


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("power", [0, 100])
def test_products_keep_the_tail(name, power):
    """h = act(g) u, and its slopes act(g) and u act'(g), with u = 2^power."""
    g = bf16_between(*SPAN[name])
    x = torch.zeros(g.numel(), 8, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = g, 2.0 ** power
    w = torch.zeros(1, 2, 8, dtype=torch.bfloat16)
    w[0, 0, 0] = w[0, 1, 1] = 1.0
    slopes = torch.empty(2, g.numel(), 1, device="cuda")
    h = ozk.grouped_gated_gemm(x.cuda(), w.cuda(), torch.tensor([0, g.numel()], dtype=torch.int32, device="cuda"),
                               activation=name, slopes=slopes)
    g, u = g.double().numpy(), 2.0 ** power
    a, p, q = exact(g, name)
    off = ref.off(g, name)
    got = [t.double().cpu().numpy().ravel() for t in (slopes[1], slopes[0], h)]
    bound = off * np.abs(a) + 2.0 ** -140
    assert np.all(np.abs(got[0] - a) <= bound)
    # two products and a sum of the slope's terms, each of P's or its derivative's error
    assert np.all(np.abs(got[1] - u * (p + q)) <= u * ((off + 6 * 2.0 ** -23) * (p + np.abs(q)) + 2.0 ** -139) + 2.0 ** -149)
    assert np.all(np.abs(got[2] - u * a) <= ref.rounded(u * bound, u * a, 2.0 ** -8, 2.0 ** -126 * 2.0 ** -8))
    assert ozk.ozk_stream_status() == 0


# In units of 2^-23: expf is off by up to 2 steps, a rounding by half a unit.  silu: e^-|g|, 1 +, the quotient, times
# e^-|g|, times g: 2 + 4 / 2.  gelu: normcdff, up to 5 steps, times g.  gelu_tanh: as silu, and z by 2 units of itself
# (its two constants, g^2, the sum and the product, half a unit each, of terms of one sign).
UNITS = {"silu": lambda z: 4.0, "gelu": lambda z: 5.5, "gelu_tanh": lambda z: 4.0 + 2 * np.abs(z)}


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("rows", [2, 4000])
def test_rows_with_4_bit_weights(name, rows):
    """act(g) in fp32 at every bf16 value of g from the span's left end to 30 (two rows: eleven of them)."""
    g = bf16_between(SPAN[name][0], 30.0)
    g = g[g.abs() >= 2.0 ** -20]
    if rows == 2:
        g = g[:: g.numel() // 10]
    w = torch.zeros(2, 64, device="cuda")
    w[0, 0] = w[1, 1] = 1.0  # MXFP4 holds a one exactly
    q = ozk.mx4_quantize(w, "mxfp4")
    x = torch.zeros(g.numel(), 64, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = g, 1.0
    x = x.cuda()
    got = torch.cat([ozk.mx4_gated_gemv(x[i: i + rows], q, activation=name, out_dtype=torch.float32)
                     for i in range(0, g.numel(), rows)])
    got, g = got.double().cpu().numpy().ravel(), g.double().numpy()
    a = exact(g, name)[0]
    z = C * (g + 0.044715 * g ** 3)
    worst = np.max((np.abs(got - a) - 2.0 ** -140) / np.abs(a)) * 2.0 ** 23
    assert np.all(np.abs(got - a) <= UNITS[name](z) * 2.0 ** -23 * np.abs(a) + 2.0 ** -140), worst
