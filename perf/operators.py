"""What the low-precision products of the library are measured on: quantisation
to microscaled 4-bit floating point, the product of two such matrices, and the
products of rows grouped by expert (16-bit operands with their gradients, and
4-bit operands).

``listed`` and ``draw`` give cases, ``prepare`` what a program holds before the
call, ``run`` one pass (the library's own calls where ``own`` is true, plain
torch operations in 32 bits otherwise), ``work`` the bytes and operations a
pass cannot do without, ``exact`` the result in 64 bits.

Storage of a 4-bit matrix of R rows and K columns (rows in G groups, group g
starting at row o_g), as the library reads and writes it: ``codes`` is uint8
[R, kp / 2], kp = K rounded up to 64, element 2i of a row in the low half of
byte i; ``scales`` is uint8 [B, kg, 32, 4, 4], the byte of row r of group g and
block b of K at [o_g // 128 + g + r // 128, b // 4, r % 32, r // 32 % 4, b % 4]
(r counted within its group), B = R // 128 + G and kg = ceil(blocks / 4).
"nvfp4" blocks hold 16 elements under an E4M3 scale, "mxfp4" blocks 32 elements
under a power of two.
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
        # one token's activations before a 4-bit layer: a launch's latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "k": 4096, "format": "nvfp4", "type": "bfloat16"},
        # a ragged batch whose rows end inside a block
        {"name": "quantize_odd", "op": "quantize", "rows": 1537, "k": 2090, "format": "mxfp4", "type": "float16"},
        # a long prompt's activations, or a layer's weights: the memory's speed
        {"name": "quantize_large", "op": "quantize", "rows": 16384, "k": 8192, "format": "nvfp4", "type": "bfloat16"},
        # one token through a 4-bit layer: the weights are read once
        {"name": "product_token", "op": "product", "m": 1, "n": 8192, "k": 4096, "format": "nvfp4", "type": "bfloat16"},
        # odd sizes in every direction, 32-bit results
        {"name": "product_odd", "op": "product", "m": 1000, "n": 1537, "k": 2090, "format": "mxfp4", "type": "float32"},
        # the largest square product of the library's own workloads
        {"name": "product_large", "op": "product", "m": 8192, "n": 8192, "k": 8192, "format": "nvfp4", "type": "bfloat16"},
        # a decoding step: a few rows, most experts get none or one
        {"name": "experts_token", "op": "experts", "rows": 16, "groups": 16, "inner": 2048, "outer": 1024,
         "type": "bfloat16", "idle": 0, "route": 1},
        # a prompt's rows through one layer of experts
        {"name": "experts_prompt", "op": "experts", "rows": 8192, "groups": 16, "inner": 4096, "outer": 2048,
         "type": "bfloat16", "idle": 0, "route": 2},
        # both gradients on odd sizes, some experts without rows
        {"name": "experts_grad_odd", "op": "experts_grad", "rows": 1999, "groups": 7, "inner": 1032, "outer": 520,
         "type": "float16", "idle": 2, "route": 3},
        # both gradients of a training step's layer
        {"name": "experts_grad_large", "op": "experts_grad", "rows": 16384, "groups": 8, "inner": 4096,
         "outer": 4096, "type": "bfloat16", "idle": 0, "route": 4},
        # a decoding step with 4-bit experts: quantise the rows, then the products
        {"name": "experts4_token", "op": "experts4", "rows": 32, "groups": 32, "inner": 4096, "outer": 2048,
         "format": "nvfp4", "type": "bfloat16", "idle": 0, "route": 5},
        # a long prompt through 4-bit experts
        {"name": "experts4_large", "op": "experts4", "rows": 16384, "groups": 16, "inner": 4096, "outer": 4096,
         "format": "mxfp4", "type": "bfloat16", "idle": 1, "route": 6},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step, step))


def draw(rng):
    op = rng.choice(["quantize", "product", "experts", "experts_grad", "experts4"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 16384), "k": _log(rng, 64, 8192), "format": fmt,
                "type": rng.choice(["bfloat16", "float16", "float32"])}
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 128, 8192), "k": _log(rng, 64, 8192),
                "format": fmt, "type": rng.choice(["bfloat16", "float32"])}
    groups = _log(rng, 2, 32)
    case = {"op": op, "rows": _log(rng, 1, 8192), "groups": groups, "inner": _log(rng, 128, 4096, 8),
            "outer": _log(rng, 128, 4096, 8), "type": rng.choice(["bfloat16", "float16"]),
            "idle": rng.choice([0, 0, groups // 4, groups // 2]), "route": rng.randrange(1 << 30)}
    if op == "experts4":
        case.update(format=fmt, type="bfloat16", inner=_log(rng, 128, 4096))
    return case


def _counts(case):
    """Rows of each expert: popular and unpopular ones, `idle` of them without any."""
    rng = np.random.RandomState(case["route"])
    g = case["groups"]
    share = rng.permutation(1.0 / np.sqrt(np.arange(1, g + 1)))
    share[rng.permutation(g)[: min(case["idle"], g - 1)]] = 0.0
    return rng.multinomial(case["rows"], share / share.sum())


def _padded(k):
    return -(-k // 64) * 64


def _scale_bytes(rows, k, fmt):
    return rows * -(-k // BLOCK[fmt])


def work(case):
    op = case["op"]
    if op == "quantize":
        r, k = case["rows"], case["k"]
        # the matrix, its codes and scales, and the values read back from them
        return {"bytes": r * k * SIZE[case["type"]] + r * k / 2 + _scale_bytes(r, k, case["format"]) + r * k * 2,
                "flops": 4 * r * k}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k / 2 + _scale_bytes(m + n, k, case["format"]) + m * n * SIZE[case["type"]],
                "flops": 2 * m * n * k}
    t, i, o, size = case["rows"], case["inner"], case["outer"], SIZE[case["type"]]
    used = int((_counts(case) > 0).sum())
    if op == "experts":
        return {"bytes": size * (t * i + used * i * o + t * o), "flops": 2 * t * i * o}
    if op == "experts_grad":
        # rows and gradients in, the weights of the experts in use, both gradients out
        return {"bytes": size * (t * i + t * o + used * i * o + t * i + case["groups"] * i * o), "flops": 4 * t * i * o}
    codes = i / 2 + _scale_bytes(1, i, case["format"])
    return {"bytes": size * t * i + t * codes + used * o * codes + size * t * o, "flops": 2 * t * i * o}


# ------------------------------------------------- plain forms, 32-bit torch
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(e):
    """2^e in 32 bits for whole -127 <= e <= 127, from its bits (exact; exp2 need not be)."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _to_scale_bytes(amax, fmt):
    """Scale bytes of blocks with largest magnitude amax, and the scales they stand for."""
    if fmt == "mxfp4":
        _, e = torch.frexp(amax)  # amax = f 2^e, f in [0.5, 1)
        e = (e - 3).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        return (e + 127).to(torch.uint8), _pow2(e)
    s = amax / 6.0
    _, e = torch.frexp(s)
    step = _pow2((e - 4).clamp(min=-9))  # spacing of E4M3 at s
    s = (torch.round(s / step) * step).clamp(max=448.0)
    _, e = torch.frexp(s)
    e = (e + 6).clamp(min=0)  # biased exponent, 0 below 2^-6
    frac = torch.where(e > 0, s * _pow2(10 - e) - 8, s * 512.0)
    return (e * 8 + frac.int()).to(torch.uint8), s


def _from_scale_bytes(b, fmt):
    b = b.int()
    if fmt == "mxfp4":
        return _pow2(b - 127)
    e, f = b >> 3, (b & 7).float()
    return torch.where(e > 0, (8 + f) * _pow2(e - 10), f / 512.0)


def _encode(x, fmt):
    """(code of every element, scale byte of every block) of the rows of x, in 32 bits."""
    rows, k = x.shape
    kp, blk = _padded(k), BLOCK[fmt]
    x = torch.nn.functional.pad(x.float(), (0, kp - k)).view(rows, kp // blk, blk)
    byte, s = _to_scale_bytes(x.abs().amax(dim=2), fmt)
    q = torch.where(s[..., None] > 0, x.abs() / s[..., None], torch.zeros_like(x))
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    code = torch.zeros_like(q, dtype=torch.uint8)
    code += (q > 0.25).byte() + (q >= 0.75).byte() + (q > 1.25).byte() + (q >= 1.75).byte()
    code += (q > 2.5).byte() + (q >= 3.5).byte() + (q > 5.0).byte()
    code += 8 * ((x < 0) & (s[..., None] > 0)).byte()
    return code.view(rows, kp), byte


def _values(code, byte, fmt):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=code.device)
    rows, kp = code.shape
    v = table[code.int()].view(rows, -1, BLOCK[fmt]) * _from_scale_bytes(byte, fmt)[..., None]
    return v.view(rows, kp)


def _places(rows, kblocks, offsets, device):
    """Where the scale byte of (row, block) lies: flat indices, and the size of the whole."""
    r = torch.arange(rows, device=device)
    g = (r[:, None] >= offsets[None, 1:-1]).sum(dim=1)
    o = offsets.long()[g]
    block = o // 128 + g + (r - o) // 128
    r = r - o
    b = torch.arange(kblocks, device=device)
    kg = -(-kblocks // 4)
    at = (block[:, None] * kg + b[None] // 4) * 512 + (r % 32 * 16 + r // 32 % 4 * 4)[:, None] + b[None] % 4
    return at, (rows // 128 + offsets.numel() - 1) * kg * 512


def _pack(x, fmt, offsets):
    """(codes, scales) of x in storage."""
    code, byte = _encode(x, fmt)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    at, size = _places(x.shape[0], byte.shape[1], offsets, x.device)
    scales = torch.zeros(size, dtype=torch.uint8, device=x.device)
    scales[at] = byte
    return codes, scales


def _unpack(codes, scales, fmt, offsets):
    """What stored (codes, scales) stand for, in 32 bits, rows padded to 64 columns."""
    rows, half = codes.shape
    code = torch.stack((codes & 15, codes >> 4), dim=2).view(rows, 2 * half)
    at, _ = _places(rows, 2 * half // BLOCK[fmt], offsets, codes.device)
    return _values(code, scales[at], fmt)


def _one_group(rows, device):
    return torch.tensor([0, rows], dtype=torch.int32, device=device)


def _even_groups(groups, rows, device):
    return torch.arange(groups + 1, dtype=torch.int32, device=device) * rows


def _spread(x, offsets, most):
    """Rows of every expert in a matrix of its own, zeros below: [groups, most, columns], and where each row went."""
    r = torch.arange(x.shape[0], device=x.device)
    g = (r[:, None] >= offsets[None, 1:-1]).sum(dim=1)
    at = g * most + r - offsets.long()[g]
    out = torch.zeros((offsets.numel() - 1) * most, x.shape[1], device=x.device)
    out[at] = x.float()
    return out.view(-1, most, x.shape[1]), at


# ------------------------------------------------------------------ the pass
def _activations(gen, rows, k, kind):
    """Activations of a layer: normal, a few columns many times larger."""
    x = torch.randn(rows, k, generator=gen, device="cuda")
    gain = torch.exp(0.4 * torch.randn(k, generator=gen, device="cuda"))
    gain = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.005, 20 * gain, gain)
    return (x * gain).to(kind)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, kind = case["op"], TYPES[case["type"]]
    state = {"case": case}
    if op == "quantize":
        state["x"] = _activations(gen, case["rows"], case["k"], kind)
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x = _activations(gen, m, k, torch.bfloat16)
        w = torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)
        state["a"] = _pack(x, case["format"], _one_group(m, "cuda"))
        state["b"] = _pack(w, case["format"], _one_group(n, "cuda"))
    else:
        t, g, i, o = case["rows"], case["groups"], case["inner"], case["outer"]
        counts = _counts(case)
        state["most"] = int(counts.max())
        state["offsets"] = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
        state["x"] = _activations(gen, t, i, kind)
        w = torch.randn(g, o, i, generator=gen, device="cuda") / math.sqrt(i)
        if op == "experts4":
            state["w"] = _pack(w.view(g * o, i), case["format"], _even_groups(g, o, "cuda"))
        else:
            state["w"] = w.to(kind)
        if op == "experts_grad":
            state["dy"] = (0.1 * torch.randn(t, o, generator=gen, device="cuda")).to(kind)
    return state


def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(state, case, case["op"], TYPES[case["type"]])


def _run_own(state, case, op, kind):
    from fp64_gemm_emulation_exponent_gb300 import ozk

    if op == "quantize":
        return ozk.mx4_dequantize(ozk.mx4_quantize(state["x"], case["format"]), torch.bfloat16)
    if op == "product":
        a = ozk.Mx4(*state["a"], case["m"], case["k"], case["format"])
        b = ozk.Mx4(*state["b"], case["n"], case["k"], case["format"])
        return ozk.mx4_gemm(a, b, out_dtype=kind)
    x, w, offsets = state["x"], state["w"], state["offsets"]
    if op == "experts":
        return ozk.grouped_gemm(x, w, offsets)
    if op == "experts_grad":
        return ozk.grouped_gemm_dx(state["dy"], w, offsets), ozk.grouped_gemm_dw(state["dy"], x, offsets)
    w = ozk.Mx4(*w, case["groups"] * case["outer"], case["inner"], case["format"], groups=case["groups"])
    return ozk.mx4_grouped_gemm(ozk.mx4_quantize(x, case["format"], offsets=offsets), w, out_dtype=kind)


def _run_plain(state, case, op, kind):
    if op == "quantize":
        x = state["x"]
        return _values(*_encode(x, case["format"]), case["format"])[:, : x.shape[1]].to(torch.bfloat16).contiguous()
    if op == "product":
        a = _unpack(*state["a"], case["format"], _one_group(case["m"], "cuda"))
        b = _unpack(*state["b"], case["format"], _one_group(case["n"], "cuda"))
        return torch.matmul(a, b.t()).to(kind)
    x, w, offsets, most = state["x"], state["w"], state["offsets"], state["most"]
    if op == "experts":
        rows, at = _spread(x, offsets, most)
        return torch.bmm(rows, w.float().transpose(1, 2)).view(-1, case["outer"])[at].to(kind)
    if op == "experts_grad":
        dys, at = _spread(state["dy"], offsets, most)
        rows, _ = _spread(x, offsets, most)
        dx = torch.bmm(dys, w.float()).view(-1, case["inner"])[at].to(kind)
        return dx, torch.bmm(dys.transpose(1, 2), rows).to(kind)
    w = _unpack(*w, case["format"], _even_groups(case["groups"], case["outer"], "cuda"))
    rows, at = _spread(_values(*_encode(x, case["format"]), case["format"]), offsets, most)
    w = w.view(case["groups"], case["outer"], -1)
    return torch.bmm(rows, w.transpose(1, 2)).view(-1, case["outer"])[at].to(kind)


# ------------------------------------------------------- from the definition
_GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _two_to(e):
    """2^e in 64 bits, e limited to a scale byte's range."""
    return torch.bitwise_left_shift(e.long().clamp(-127, 127) + 1023, 52).view(torch.float64)


def _exact_values(x, fmt):
    """The 4-bit values of x's rows: the scale from the format's rule, every element the nearest grid point (of two
    equally near ones that with the even code), in 64 bits."""
    rows, k = x.shape
    blk = BLOCK[fmt]
    x = torch.cat((x.double(), x.new_zeros(rows, -k % blk).double()), dim=1).view(rows, -1, blk)
    top = x.abs().max(dim=2, keepdim=True).values
    if fmt == "mxfp4":
        _, e = torch.frexp(top)  # top = f 2^e, 1/2 <= f < 1
        s = torch.where(top > 0, _two_to(e - 3), 0.0)
    else:
        grid = torch.tensor([m * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8, 16)][:-1], dtype=torch.float64)
        grid = torch.cat((torch.arange(8, dtype=torch.float64) / 512, grid)).to(x.device)
        s = grid[_nearest(grid, top / 6.0)]
    q = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    grid = _GRID.to(x.device)
    v = grid[_nearest(grid, q)] * s * torch.sign(x)
    return v.view(rows, -1)[:, :k]


def _nearest(grid, q):
    up = torch.searchsorted(grid, q.contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = q - grid[up - 1], grid[up] - q
    return torch.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)


def _stored_values(codes, scales, k, fmt, group_rows):
    """Stored 4-bit rows (groups of group_rows) as 64-bit values."""
    rows, blk = codes.shape[0], BLOCK[fmt]
    both = torch.stack((codes % 16, codes // 16), dim=2).reshape(rows, -1)[:, :k].long()
    v = _GRID.to(codes.device)[both % 8] * torch.where(both >= 8, -1.0, 1.0).double()
    kg = -(-(-(-_padded(k) // blk)) // 4)
    row = torch.arange(rows, device=codes.device)
    g, r = row // group_rows, row % group_rows
    tile = g * group_rows // 128 + g + r // 128
    byte = scales.view(-1, kg, 32, 4, 4)[tile, :, r % 32, r // 32 % 4].reshape(rows, -1).double()
    if fmt == "mxfp4":
        s = _two_to(byte - 127)
    else:
        e, f = torch.floor(byte / 8), byte % 8
        s = torch.where(e > 0, (1 + f / 8) * _two_to(e - 7), f * 2.0 ** -9)
    return v * s.repeat_interleave(blk, dim=1)[:, :k]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(state["x"], case["format"])
    if op == "product":
        a = _stored_values(*state["a"], case["k"], case["format"], case["m"])
        b = _stored_values(*state["b"], case["k"], case["format"], case["n"])
        return torch.einsum("mk,nk->mn", a, b)
    x, ends = state["x"].double(), np.cumsum(_counts(case)).tolist()
    spans = [(g, lo, hi) for g, (lo, hi) in enumerate(zip([0] + ends[:-1], ends))]
    if op == "experts_grad":
        w, dy = state["w"].double(), state["dy"].double()
        return (torch.cat([dy[lo:hi] @ w[g] for g, lo, hi in spans]),
                torch.stack([dy[lo:hi].t() @ x[lo:hi] for _, lo, hi in spans]))
    if op == "experts4":
        x = _exact_values(state["x"], case["format"])
        w = _stored_values(*state["w"], case["inner"], case["format"], case["outer"])
        w = w.view(case["groups"], case["outer"], case["inner"])
    else:
        w = state["w"].double()
    return torch.cat([x[lo:hi] @ w[g].t() for g, lo, hi in spans])


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(c, work(c))
