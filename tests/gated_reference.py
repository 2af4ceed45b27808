"""The gated product in 64 bits, for the tests, and how far the kernels may be off.

Let g and u be the two projections.  The kernels sum K terms in fp32: each of
the K additions is off by at most 2^-23 of the magnitudes summed so far, so
dg <= K 2^-23 sum |x w|, and du alike.  act(g) = g P(g), and P's error comes
from its exponential e^z, z = g (silu), g^2 / 2 (gelu) or 2 sqrt(2 / pi) (g +
0.044715 g^3) (gelu_tanh): z is rounded up to three times (half a unit of 2^-23
each, relative, so e^z is off by 1.5 |z| units), the exponential itself by 2 + 1.2
|z| units, and what follows (a sum, a quotient, a polynomial fitted to 5e-7, a
product) by up to 10: off(z) = 12 + 2.7 |z| units.  Up to |z| = 19 that is at most
64 units, 2^-17 of act(g); beyond, |act(g)| on the left is below 20 e^-19 = 2^-23
and falls faster than off(z) grows, so that 2^-23 times 64 units, 2^-40, covers it.
|act'| <= 1.13 and |act''| <= 1.13 for all three."""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[float])
ACTS = ("silu", "gelu", "gelu_tanh")


def act(g, name):
    """(act(g), act'(g))."""
    if name == "gelu":
        p = 0.5 * (1 + _erf(g * math.sqrt(0.5)))
        return g * p, p + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(8 / math.pi)
    z, dz = (g, 1.0) if name == "silu" else (c * (g + 0.044715 * g ** 3), c * (1 + 0.134145 * g * g))
    e = np.exp(-np.abs(z))
    p = np.where(z >= 0, 1, e) / (1 + e)
    return g * p, p + g * (e / (1 + e) ** 2) * dz


def off(g, name):
    """The relative error of P(g), see above."""
    z = {"silu": g, "gelu": g * g / 2, "gelu_tanh": math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)}[name]
    return (12 + 2.7 * np.abs(z)) * 2.0 ** -23


class Gated:
    """h, its slopes and the bounds on their errors before rounding, for one group's rows."""

    def __init__(self, x, w, name, scale=1.0, extra=0):
        H = w.shape[0] // 2
        pre, err = scale * (x @ w.T), (x.shape[1] + extra) * 2.0 ** -23 * abs(scale) * (np.abs(x) @ np.abs(w).T)
        g, u, dg, du = pre[:, :H], pre[:, H:], err[:, :H], err[:, H:]
        a, s = act(g, name)
        da = 1.13 * dg + 2.0 ** -17 * np.abs(a) + 2.0 ** -40
        ds = 1.13 * dg + 2.0 ** -16
        self.h, self.dh = a * u, da * np.abs(u) + (np.abs(a) + da) * du
        self.by_gate, self.d_gate = u * s, ds * np.abs(u) + (np.abs(s) + ds) * du
        self.by_up, self.d_up = a, da


def rounded(bound, exact, half, least):
    """`bound` and the rounding to a type of half a step `half` (relative), `least` in absolute terms."""
    return bound + half * (np.abs(exact) + bound) + least
