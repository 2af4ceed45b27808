"""What the gated feed-forward products of the library are measured on: the
gated product of rows grouped by expert (both projections, the activation and
their product), a training step of it with its gradients, and the products of a
few 16-bit rows with 4-bit weights, plain and gated.

``listed`` and ``draw`` give cases, ``prepare`` what a program holds before the
call, ``run`` one pass (the library's own calls where ``own`` is true, plain
torch operations in 32 bits otherwise), ``work`` the bytes and operations a
pass cannot do without, ``exact`` the result in 64 bits.

A gated product: rows x_t of expert e, weights w_e of 2 H rows, the gate's
first: h_t = act(x_t w_e[:H]^T) * (x_t w_e[H:]^T).

Storage of a 4-bit matrix of G equal groups of R rows and K columns: ``codes``
is uint8 [G R, kp / 2], kp = K rounded up to 64, element 2i of a row in the low
half of byte i; ``scales`` is uint8, the byte of row r of group g and block b of
K at [g R // 128 + g + r // 128, b // 4, r % 32, r // 32 % 4, b % 4] of a
[.., ceil(blocks / 4), 32, 4, 4] array.  "nvfp4" blocks hold 16 elements under
an E4M3 scale, "mxfp4" blocks 32 elements under a power of two.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32}
TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
SIZE = {"bfloat16": 2, "float16": 2, "float32": 4}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decoding step of a layer of experts: most get none or one of the rows
        {"name": "gated_token", "op": "gated", "rows": 16, "groups": 16, "inner": 2048, "outer": 1024,
         "type": "bfloat16", "act": "silu", "idle": 0, "route": 1},
        # a ragged batch on odd sizes, some experts without rows
        {"name": "gated_odd", "op": "gated", "rows": 1999, "groups": 7, "inner": 1032, "outer": 520,
         "type": "float16", "act": "gelu", "idle": 2, "route": 2},
        # a prompt's rows through one layer of experts
        {"name": "gated_prompt", "op": "gated", "rows": 8192, "groups": 16, "inner": 4096, "outer": 2048,
         "type": "bfloat16", "act": "silu", "idle": 0, "route": 3},
        # a small training step on odd sizes, one expert without rows
        {"name": "gated_train_odd", "op": "gated_train", "rows": 1537, "groups": 5, "inner": 520, "outer": 1032,
         "type": "float16", "act": "gelu_tanh", "idle": 1, "route": 4},
        # a training step's layer: the product and both gradients
        {"name": "gated_train_large", "op": "gated_train", "rows": 16384, "groups": 8, "inner": 4096, "outer": 4096,
         "type": "bfloat16", "act": "silu", "idle": 0, "route": 5},
        # one token through a 4-bit layer: the weights are read once
        {"name": "gemv_token", "op": "gemv", "rows": 1, "groups": 1, "inner": 4096, "outer": 8192,
         "format": "nvfp4", "type": "bfloat16", "result": "bfloat16", "idle": 0, "route": 6},
        # a few rows, odd sizes in every direction, 32-bit results
        {"name": "gemv_odd", "op": "gemv", "rows": 5, "groups": 1, "inner": 2090, "outer": 1537,
         "format": "mxfp4", "type": "float16", "result": "float32", "idle": 0, "route": 7},
        # a batch of requests, one token each
        {"name": "gemv_batch", "op": "gemv", "rows": 16, "groups": 1, "inner": 8192, "outer": 8192,
         "format": "nvfp4", "type": "bfloat16", "result": "bfloat16", "idle": 0, "route": 8},
        # a decoding step of 4-bit experts, the second product
        {"name": "gemv_experts", "op": "gemv", "rows": 32, "groups": 32, "inner": 4096, "outer": 2048,
         "format": "mxfp4", "type": "bfloat16", "result": "bfloat16", "idle": 0, "route": 9},
        # one token through both projections of a 4-bit gated layer
        {"name": "gated_gemv_token", "op": "gated_gemv", "rows": 1, "groups": 1, "inner": 4096, "outer": 8192,
         "format": "nvfp4", "type": "bfloat16", "result": "bfloat16", "act": "silu", "idle": 0, "route": 10},
        # a decoding step of 4-bit experts, the gated product
        {"name": "gated_gemv_experts", "op": "gated_gemv", "rows": 16, "groups": 16, "inner": 4096, "outer": 2048,
         "format": "nvfp4", "type": "bfloat16", "result": "bfloat16", "act": "gelu_tanh", "idle": 4, "route": 11},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step, step))


def draw(rng):
    op = rng.choice(["gated", "gated_train", "gemv", "gated_gemv"])
    case = {"op": op, "type": rng.choice(["bfloat16", "float16"]), "route": rng.randrange(1 << 30)}
    if op in ("gated", "gated_train"):
        groups = _log(rng, 1, 32)
        case.update(rows=_log(rng, 1, 8192), groups=groups, inner=_log(rng, 128, 4096, 8), outer=_log(rng, 128, 4096, 8))
    else:
        groups = rng.choice([1, _log(rng, 2, 32)])
        case.update(rows=_log(rng, 1, 32), groups=groups, inner=_log(rng, 64, 8192),
                    outer=_log(rng, 128, 16384 if groups == 1 else 4096), format=rng.choice(["nvfp4", "mxfp4"]))
        case["result"] = rng.choice([case["type"], "float32"])
    if op != "gemv":
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
    case["idle"] = rng.choice([0, 0, groups // 4, groups // 2])
    return case


def _counts(case):
    """Rows of each expert: popular and unpopular ones, `idle` of them without any."""
    rng = np.random.RandomState(case["route"])
    g = case["groups"]
    share = rng.permutation(1.0 / np.sqrt(np.arange(1, g + 1)))
    share[rng.permutation(g)[: min(case["idle"], g - 1)]] = 0.0
    return rng.multinomial(case["rows"], share / share.sum())


def work(case):
    op, t, i, o, size = case["op"], case["rows"], case["inner"], case["outer"], SIZE[case["type"]]
    used = int((_counts(case) > 0).sum())
    if op == "gated":
        return {"bytes": size * (t * i + used * 2 * o * i + t * o), "flops": 4 * t * i * o}
    if op == "gated_train":
        # rows, weights in use and the result's gradient in; the result and both gradients out
        return {"bytes": size * (2 * t * i + 2 * t * o + (used + case["groups"]) * 2 * o * i), "flops": 12 * t * i * o}
    n = o if op == "gemv" else 2 * o
    weights = used * n * (i / 2 + -(-i // BLOCK[case["format"]]))
    return {"bytes": size * t * i + weights + SIZE[case["result"]] * t * o, "flops": 2 * t * i * n}


# ------------------------------------------------------------------ the inputs
def _activations(gen, rows, k, kind):
    """Activations of a layer: normal, a few columns many times larger."""
    x = torch.randn(rows, k, generator=gen, device="cuda")
    gain = torch.exp(0.4 * torch.randn(k, generator=gen, device="cuda"))
    gain = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.005, 20 * gain, gain)
    return (x * gain).to(kind)


def _places(groups, rows, blocks, device):
    """Where the scale byte of (group, row, block) lies: flat indices [groups, rows, blocks], and the size of the whole."""
    g = torch.arange(groups, device=device)[:, None, None]
    r = torch.arange(rows, device=device)[None, :, None]
    b = torch.arange(blocks, device=device)[None, None, :]
    words = -(-blocks // 4)
    tile = g * rows // 128 + g + r // 128
    return (tile * words + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4, (groups * rows // 128 + groups) * words * 512


def _stored(w, fmt):
    """(codes, scales, factor) of the weights w [groups, rows, k]: 4-bit storage, scaled by a power of two into the
    block scales' range; the factor takes it back."""
    groups, rows, k = w.shape
    blk, kp = BLOCK[fmt], -(-k // 64) * 64
    scale = 2.0 ** math.floor(math.log2(6 * 448 / float(w.abs().max()))) if fmt == "nvfp4" else 1.0
    v = torch.nn.functional.pad(w * scale, (0, kp - k)).view(groups, rows, kp // blk, blk)
    top = v.abs().amax(dim=3)
    if fmt == "nvfp4":
        s8 = (top / 6.0).to(torch.float8_e4m3fn)
        byte, s = s8.view(torch.uint8), s8.float()
    else:
        e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
        byte, s = (e + 127).to(torch.uint8), torch.exp2(e.float())
    q = torch.where(s[..., None] > 0, v.abs() / s[..., None], 0.0)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(q, edges).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
    code = code.view(groups * rows, kp)
    at, size = _places(groups, rows, kp // blk, w.device)
    scales = torch.zeros(size, dtype=torch.uint8, device=w.device)
    scales[at.flatten()] = byte.flatten()
    return code[:, 0::2] | (code[:, 1::2] << 4), scales, 1.0 / scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, kind = case["op"], TYPES[case["type"]]
    t, g, i, o = case["rows"], case["groups"], case["inner"], case["outer"]
    counts = _counts(case)
    state = {"case": case, "most": int(counts.max()), "x": _activations(gen, t, i, kind)}
    state["offsets"] = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
    w = torch.randn(g, o if op == "gemv" else 2 * o, i, generator=gen, device="cuda") / math.sqrt(i)
    if op in ("gemv", "gated_gemv"):
        state["codes"], state["scales"], state["alpha"] = _stored(w, case["format"])
        return state
    state["w"] = w.to(kind)
    if op == "gated_train":
        state["dh"] = (0.1 * torch.randn(t, o, generator=gen, device="cuda")).to(kind)
        state["x"].requires_grad_()
        state["w"].requires_grad_()
    return state


# ------------------------------------------------------------------ the pass
def run(state):
    case = state["case"]
    return _run_own(state, case, case["op"]) if own else _run_plain(state, case, case["op"])


def _run_own(state, case, op):
    from fp64_gemm_emulation_exponent_gb300 import ozk

    x, offsets = state["x"], state["offsets"]
    if op == "gated":
        return ozk.grouped_gated_gemm(x, state["w"], offsets, activation=case["act"])
    if op == "gated_train":
        h = ozk.grouped_gated_gemm(x, state["w"], offsets, activation=case["act"])
        dx, dw = torch.autograd.grad(h, (x, state["w"]), state["dh"])
        return h.detach(), dx, dw
    rows = case["outer"] * (1 if op == "gemv" else 2)
    w = ozk.Mx4(state["codes"], state["scales"], case["groups"] * rows, case["inner"], case["format"],
                groups=case["groups"])
    offsets = None if case["groups"] == 1 else offsets
    if op == "gemv":
        return ozk.mx4_gemv(x, w, offsets, alpha=state["alpha"], out_dtype=TYPES[case["result"]])
    return ozk.mx4_gated_gemv(x, w, offsets, activation=case["act"], alpha=state["alpha"],
                              out_dtype=TYPES[case["result"]])


def _spread(x, offsets, most):
    """Rows of every expert in a matrix of its own, zeros below: [groups, most, columns], and where each row went."""
    r = torch.arange(x.shape[0], device=x.device)
    g = (r[:, None] >= offsets[None, 1:-1]).sum(dim=1)
    at = g * most + r - offsets.long()[g]
    out = torch.zeros((offsets.numel() - 1) * most, x.shape[1], device=x.device)
    out[at] = x.float()
    return out.view(-1, most, x.shape[1]), at


def _unpack(state, fmt, groups):
    """What stored weights stand for, in 32 bits: [groups, rows, padded columns]."""
    codes = state["codes"]
    code = torch.stack((codes & 15, codes >> 4), dim=2).view(groups, -1, 2 * codes.shape[1])
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat((table, -table))
    at, _ = _places(groups, code.shape[1], code.shape[2] // BLOCK[fmt], codes.device)
    byte = state["scales"][at]
    s = byte.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else (byte.int() << 23).view(torch.float32)
    return (table[code.int()].view(*s.shape, BLOCK[fmt]) * s[..., None]).view(code.shape)


_SQRT_2_PI = math.sqrt(2 / math.pi)


def _act(g, act):
    """(act(g), its derivative)."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (0.5 * _SQRT_2_PI)
    t = torch.tanh(_SQRT_2_PI * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * (_SQRT_2_PI * (1 + 0.134145 * g * g))


@torch.no_grad()
def _run_plain(state, case, op):
    offsets, o = state["offsets"], case["outer"]
    rows, at = _spread(state["x"], offsets, state["most"])
    if op in ("gemv", "gated_gemv"):
        w = _unpack(state, case["format"], case["groups"])[:, :, : case["inner"]]
        y = torch.bmm(rows, w.transpose(1, 2)).view(-1, w.shape[1])[at] * state["alpha"]
        if op == "gated_gemv":
            y = _act(y[:, :o], case["act"])[0] * y[:, o:]
        return y.to(TYPES[case["result"]])
    kind, w = TYPES[case["type"]], state["w"].float()
    pre = torch.bmm(rows, w.transpose(1, 2))
    a, slope = _act(pre[:, :, :o], case["act"])
    h = (a * pre[:, :, o:]).view(-1, o)[at].to(kind)
    if op == "gated":
        return h
    dh, _ = _spread(state["dh"], offsets, state["most"])
    dpre = torch.cat((dh * pre[:, :, o:] * slope, dh * a), dim=2)
    dx = torch.bmm(dpre, w).view(-1, case["inner"])[at].to(kind)
    return h, dx, torch.bmm(dpre.transpose(1, 2), rows).to(kind)


# ------------------------------------------------------- from the definition
def _weights_64(state, case, n):
    """Stored 4-bit weights as 64-bit values [groups, n, k]."""
    k, fmt, groups = case["inner"], case["format"], case["groups"]
    codes, scales = state["codes"], state["scales"]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    both = torch.stack((codes % 16, codes // 16), dim=2).reshape(groups * n, -1)[:, :k].long()
    v = torch.where(both >= 8, -grid[both % 8], grid[both % 8])
    blocks = -(-k // 64) * 64 // BLOCK[fmt]
    row = torch.arange(groups * n, device=codes.device)
    g, r = row // n, row % n
    byte = scales.view(-1, -(-blocks // 4), 32, 4, 4)[g * n // 128 + g + r // 128, :, r % 32, r // 32 % 4]
    byte = byte.reshape(groups * n, -1).double()
    if fmt == "mxfp4":
        s = torch.ldexp(torch.ones_like(byte), byte - 127)
    else:
        e, f = torch.floor(byte / 8), byte % 8
        s = torch.where(e > 0, torch.ldexp(8 + f, e - 10), f / 512)
    return (v * s.repeat_interleave(BLOCK[fmt], dim=1)[:, :k]).view(groups, n, k)


def _gate_64(g, act):
    """(act(g), its derivative) in 64 bits: g P(g) with P a logistic function, the normal distribution's or the
    latter's approximation by tanh, which is a logistic function of twice its argument."""
    if act == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    z, dz = (g, torch.ones_like(g)) if act == "silu" else (
        math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3), math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g ** 2))
    p = torch.sigmoid(z)
    return g * p, p + g * p * torch.sigmoid(-z) * dz


@torch.no_grad()
def exact(case, seed):
    state = prepare(case, seed)
    op, o = case["op"], case["outer"]
    x, ends = state["x"].double(), np.cumsum(_counts(case)).tolist()
    spans = [(g, lo, hi) for g, (lo, hi) in enumerate(zip([0] + ends[:-1], ends))]
    if op in ("gemv", "gated_gemv"):
        w = _weights_64(state, case, o if op == "gemv" else 2 * o) * state["alpha"]
    else:
        w = state["w"].double()
    pre = torch.cat([x[lo:hi] @ w[g].t() for g, lo, hi in spans])
    if op == "gemv":
        return pre
    value, slope = _gate_64(pre[:, :o], case["act"])
    h = value * pre[:, o:]
    if op != "gated_train":
        return h
    dh = state["dh"].double()
    dpre = torch.cat((dh * slope * pre[:, o:], dh * value), dim=1)
    return (h, torch.cat([dpre[lo:hi] @ w[g] for g, lo, hi in spans]),
            torch.stack([dpre[lo:hi].t() @ x[lo:hi] for _, lo, hi in spans]))


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(c, work(c))
