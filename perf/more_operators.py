"""Measured cases of the operators of a gated feed-forward block in MXFP8.

Five operators, each in its plain form (elementary torch operations in 32 bits)
and through this package's entry points:

- ``norm``, forward: the residual's addition, the root-mean-square norm of the
  sum and the norm's output as MX copies (what the products after it read).
- ``norm``, backward: the gradient of the sum from the norm's and the residual
  stream's, the weight's gradient, and the MX copies of the first (the dY of the
  product whose output was added).
- ``product``: both projections of a gated feed-forward block, the activation
  and the product of the two in one call, optionally keeping the projections.
- ``gate``, forward: activation and product from kept projections, as MX copies
  (what the down projection reads), dense or in the experts' segments.
- ``gate``, backward: the projections' gradients as MX copies.

An MX copy comes back as its E4M3 codes (the values that they stand for under
their scales) and its E8M0 scales in the layout that the products read.

A case is a dict of plain values. Both forms take what prepare() gives.
"""

import math
import random

import torch

own = False

DEV = "cuda"
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
ROW, COL = 1, 2                       # the copies of "axis": 1x32 blocks along rows, 32x1 blocks down columns


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One token of a model in use, before its feed-forward block: only the row copy is read. Latency counts.
        {"name": "norm fwd one token", "op": "norm", "dir": "fwd", "rows": 1, "cols": 2048, "pad": 0, "res": "bf16",
         "axis": 1, "keep": False},
        # The norm before a block's projections at 16384 tokens, both copies for forward and weight gradient.
        {"name": "norm fwd 16384x2048", "op": "norm", "dir": "fwd", "rows": 16384, "cols": 2048, "pad": 0, "res": "bf16",
         "axis": 3, "keep": False},
        # The quantiser sweep's width with the residual stream in FP32, the norm's output kept in BF16 too (a router reads it).
        {"name": "norm fwd 8192x7168", "op": "norm", "dir": "fwd", "rows": 8192, "cols": 7168, "pad": 0, "res": "f32",
         "axis": 3, "keep": True},
        # Its backward pass at 16384 tokens: the gradient goes on in the stream and, as copies, into the product before.
        {"name": "norm bwd 16384x2048", "op": "norm", "dir": "bwd", "rows": 16384, "cols": 2048, "pad": 0, "res": "bf16",
         "axis": 3, "keep": False},
        # A short batch of odd length with a row pitch, FP32 stream, no copies.
        {"name": "norm bwd 1001x1408", "op": "norm", "dir": "bwd", "rows": 1001, "cols": 1408, "pad": 8, "res": "f32",
         "axis": 0, "keep": False},
        # One token through the dense FFN's two projections: the weights' bytes, latency counts.
        {"name": "product one token", "op": "product", "m": 1, "f": 10944, "k": 2048, "act": "silu", "keep": False},
        # The dense FFN's projections in training, both kept for the backward pass.
        {"name": "product 8192x10944", "op": "product", "m": 8192, "f": 10944, "k": 2048, "act": "silu", "keep": True},
        # An expert's width with an odd number of tokens, GELU.
        {"name": "product 333x1408", "op": "product", "m": 333, "f": 1408, "k": 2048, "act": "gelu", "keep": True},
        # Short batch through one expert's width: latency counts.
        {"name": "gate fwd 512x1408", "op": "gate", "dir": "fwd", "rows": 512, "f": 1408, "groups": 0, "act": "silu", "axis": 3},
        # 64 routed experts, uneven and some empty, the down projection's operands.
        {"name": "gate fwd 64 experts", "op": "gate", "dir": "fwd", "rows": 49152, "f": 1408, "groups": 64, "act": "silu",
         "axis": 3},
        # The dense FFN's backward pass.
        {"name": "gate bwd 8192x10944", "op": "gate", "dir": "bwd", "rows": 8192, "f": 10944, "groups": 0, "act": "silu",
         "axis": 3},
        # The routed experts' backward pass.
        {"name": "gate bwd 64 experts", "op": "gate", "dir": "bwd", "rows": 49152, "f": 1408, "groups": 64, "act": "silu",
         "axis": 3},
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "product", "gate", "gate"])
    if op == "norm":
        cols = 32 * _log(rng, 1, 512)
        rows = _log(rng, 1, min(65536, 50_000_000 // cols))
        back = rng.random() < 0.5
        axis = rng.choice([0, 1, 3, 3] if back else [1, 3, 3])
        if axis == 3:
            rows = max(32, rows // 32 * 32)
        return {"op": op, "dir": "bwd" if back else "fwd", "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 8, 64]),
                "res": rng.choice(["bf16", "bf16", "f32"]), "axis": axis, "keep": (not back) and rng.random() < 0.3}
    act = rng.choice(["silu", "silu", "gelu", "relu", "none"])
    f = 32 * _log(rng, 1, 342)
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 8192), "f": f, "k": 32 * _log(rng, 1, 64), "act": act, "keep": rng.random() < 0.5}
    groups = _log(rng, 1, 128) if rng.random() < 0.5 else 0
    axis = rng.choice([1, 3, 3])
    rows = _log(rng, 1, min(65536, 60_000_000 // f))
    if axis == 3 and not groups:
        rows = max(32, rows // 32 * 32)
    return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "rows": rows, "f": f, "groups": groups, "act": act, "axis": axis}


def work(case):
    op = case["op"]
    if op == "product":
        m, f, k = case["m"], case["f"], case["k"]
        return {"bytes": (m + 2 * f) * (k + k // 32) + 2 * m * f * (3 if case["keep"] else 1), "flops": 4 * m * f * k}
    copies = bin(case["axis"]).count("1") * (1 + 1 / 32)
    if op == "norm":
        r, c, s = case["rows"], case["cols"], 4 if case["res"] == "f32" else 2
        if case["dir"] == "fwd":
            return {"bytes": r * c * (2 + 2 * s + copies + 2 * case["keep"]) + 4 * c + 4 * r, "flops": 6 * r * c}
        return {"bytes": r * c * (2 + 3 * s + copies) + 8 * c + 4 * r, "flops": 12 * r * c}
    n = case["rows"] * case["f"]
    if case["dir"] == "fwd":
        return {"bytes": n * (4 + copies), "flops": 8 * n}
    return {"bytes": n * (6 + 2 * copies), "flops": 16 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen, device=DEV, dtype=F32) * std).to(dtype)


def prepare(case, seed):
    return {"norm": _prepare_norm, "product": _prepare_product, "gate": _prepare_gate}[case["op"]](case, seed)


def _prepare_norm(case, seed):
    """A residual stream some of whose columns are much larger than the rest, and
    the output of a product that is added to it."""
    gen = _rng(seed)
    r, c, dt = case["rows"], case["cols"], DTYPES[case["res"]]
    loud = torch.where(torch.rand(c, generator=gen, device=DEV) < 0.01, 20.0, 1.0)

    def rows(std, dtype):
        x = torch.empty(r, c + case["pad"], device=DEV, dtype=dtype)[:, :c]
        return x.copy_(_normal(gen, r, c) * std)

    s = {"case": case, "weight": 1.0 + _normal(gen, c, std=0.1)}
    if case["dir"] == "fwd":
        s["x"], s["residual"] = rows(0.5, BF16), rows(2.0 * loud, dt)
    else:
        s["sum"], s["dy"], s["dsum"] = rows(2.0 * loud, dt), rows(0.01, BF16), rows(0.02, dt)
        s["rstd"] = 1.0 / torch.sqrt(s["sum"].to(F32).square().mean(1) + EPS)
    return s


def _prepare_product(case, seed):
    """Quantised tokens and weights as the quantiser lays them out."""
    gen = _rng(seed)
    m, f, k = case["m"], case["f"], case["k"]
    return {"case": case, "a": _mx_rows(_normal(gen, m, k)),
            "gate": _mx_rows(_normal(gen, f, k, std=1.0 / math.sqrt(k))), "up": _mx_rows(_normal(gen, f, k, std=1.0 / math.sqrt(k)))}


def _counts(rows, groups):
    """Tokens of each expert: popularity falls with rank, every eighth expert has none."""
    r = random.Random(rows * 1009 + groups)
    share = [0.0 if e % 8 == 7 else 1.0 / (e + 1) for e in range(groups)]
    r.shuffle(share)
    total = sum(share)
    n = [int(rows * x / total) for x in share]
    n[max(range(groups), key=lambda e: share[e])] += rows - sum(n)
    return n


def _prepare_gate(case, seed):
    """The two projections side by side (gate, then up), and the gradient that the
    down projection hands back."""
    gen = _rng(seed)
    r, f = case["rows"], case["f"]
    s = {"case": case, "gate_up": _normal(gen, r, 2 * f, dtype=BF16), "offsets": None, "capacity": r}
    if case["groups"]:
        n = _counts(r, case["groups"])
        s["offsets"] = torch.tensor([sum(n[:e]) for e in range(len(n) + 1)], dtype=torch.int64).to(DEV)
        s["capacity"] = sum(-(-x // 128) * 128 for x in n)
    if case["dir"] == "bwd":
        s["dh"] = _normal(gen, r, f, std=0.01, dtype=BF16)
    return s


# ---------------------------------------------------------------------------
# MX copies in torch
# ---------------------------------------------------------------------------

def _atoms(exp):
    """Scale exponents [R, K/32] as E8M0 codes in atoms of 128 rows x 4 blocks of 32 (zero bytes past the ends)."""
    r, kb = exp.shape
    ra, ka = -(-r // 128), -(-kb // 4)
    grid = torch.zeros(ra * 128, ka * 4, dtype=torch.uint8, device=exp.device)
    grid[:r, :kb] = (exp + 127).to(torch.uint8)
    return grid.view(ra, 4, 32, ka, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _mx_rows(x):
    """E4M3 codes [R, K] under one power of two for 32 of a row, and those scales."""
    r, k = x.shape
    blocks = x.view(r, k // 32, 32)
    top = blocks.abs().amax(2)
    exp = torch.where(top > 0, torch.frexp(top).exponent - 1 - 8, -127).clamp(-127, 127)
    codes = (blocks * torch.exp2(-exp.to(F32))[..., None]).clamp(-448, 448).to(E4M3).view(r, k)
    return codes, _atoms(exp)


def _mx_values(copy, rows, dtype=F32):
    codes, atoms = copy
    k = codes.shape[1]
    ra, ka = -(-rows // 128), -(-(k // 32) // 4)
    grid = atoms.view(ra, ka, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(ra * 128, ka * 4)[:rows, :k // 32]
    return (codes.to(dtype).view(rows, k // 32, 32) * torch.exp2(grid.to(dtype) - 127)[..., None]).view(rows, k)


def _segments(x, offsets, capacity):
    """Rows of x at the places of the experts' segments, each padded with zeros to a multiple of 128."""
    counts = offsets[1:] - offsets[:-1]
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    at = torch.arange(capacity, device=x.device)
    e = torch.searchsorted(ends, at, right=True)
    row = at - (ends[e] - (counts[e] + 127) // 128 * 128)
    inside = row < counts[e]
    return torch.where(inside[:, None], x[torch.where(inside, offsets[e] + row, 0)], 0.0)


def _copies(y, s):
    """What the quantised outputs hold, of FP32 values y: the copies that the case asks for."""
    out = {}
    if s["case"]["axis"] & ROW:
        out["row"], out["row_scale"] = _mx_rows(y)
        out["row_scale"] = out["row_scale"].view(E8M0)
    if s["case"]["axis"] & COL:
        if s.get("offsets") is not None:
            y = _segments(y, s["offsets"], s["capacity"])
        out["col"], out["col_scale"] = _mx_rows(y.t().contiguous())
        out["col_scale"] = out["col_scale"].view(E8M0)
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op, back = state["case"]["op"], state["case"].get("dir") == "bwd"
    if op == "norm":
        if back:
            return (_own_norm_backward if own else _plain_norm_backward)(state)
        return (_own_norm_forward if own else _plain_norm_forward)(state)
    if op == "product":
        return (_own_product if own else _plain_product)(state)
    if back:
        return (_own_gate_backward if own else _plain_gate_backward)(state)
    return (_own_gate_forward if own else _plain_gate_forward)(state)


# The framework's calls ------------------------------------------------------

def _held(row, col):
    out = {}
    if row is not None:
        out["row"], out["row_scale"] = row.data.view(E4M3), row.scale.view(E8M0)
    if col is not None:
        out["col"], out["col_scale"] = col.data.view(E4M3), col.scale.view(E8M0)
    return out


def _own_norm_forward(s):
    import mxfp8_block_scaled_gb300 as mx
    c = s["case"]
    n = mx.add_norm_quantize(s["x"], s["residual"], s["weight"], eps=EPS, axis=c["axis"], keep_output=c["keep"])
    out = {"sum": n.sum, "rstd": n.rstd, **_held(n.row, n.col)}
    return {**out, "y": n.y} if c["keep"] else out


def _own_norm_backward(s):
    import mxfp8_block_scaled_gb300 as mx
    g = mx.add_norm_backward(s["dy"], s["sum"], s["weight"], s["rstd"], dsum=s["dsum"], axis=s["case"]["axis"])
    return {"dx": g.dx, "dweight": g.dweight, **_held(g.row, g.col)}


def _own_product(s):
    import mxfp8_block_scaled_gb300 as mx
    c = s["case"]
    a, gate, up = (mx.MXTensor(s[n][0].view(torch.uint8), s[n][1], s[n][0].shape[0], c["k"], mx.MX_ROWWISE) for n in ("a", "gate", "up"))
    out, gate_up = mx.gemm_gated(a, gate, up, act=c["act"], keep_preact=c["keep"])
    return {"out": out, "gate_up": gate_up} if c["keep"] else {"out": out}


def _own_gate_forward(s):
    import mxfp8_block_scaled_gb300 as mx
    c = s["case"]
    return _held(*mx.gated_quantize(s["gate_up"], act=c["act"], axis=c["axis"], group_offsets=s["offsets"],
                                    col_capacity=s["capacity"] if c["groups"] else None))


def _own_gate_backward(s):
    import mxfp8_block_scaled_gb300 as mx
    c = s["case"]
    return _held(*mx.gated_backward_quantize(s["dh"], s["gate_up"], act=c["act"], axis=c["axis"], group_offsets=s["offsets"],
                                             col_capacity=s["capacity"] if c["groups"] else None))


# The plain forms ------------------------------------------------------------

def _plain_norm_forward(s):
    v = s["x"].to(F32) + s["residual"].to(F32)
    rstd = 1.0 / torch.sqrt(v.square().mean(1) + EPS)
    y = v * rstd[:, None] * s["weight"]
    out = {"sum": v.to(s["residual"].dtype), "rstd": rstd, **_copies(y, s)}
    return {**out, "y": y.to(BF16)} if s["case"]["keep"] else out


def _plain_norm_backward(s):
    dy, rstd = s["dy"].to(F32), s["rstd"][:, None]
    h = s["sum"].to(F32) * rstd
    g = dy * s["weight"]
    dx = s["dsum"].to(F32) + rstd * (g - h * (g * h).mean(1, keepdim=True))
    return {"dx": dx.to(s["sum"].dtype), "dweight": (dy * h).sum(0), **_copies(dx, s)}


GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        t = torch.tanh(GELU_A * (z + GELU_B * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_A * (1.0 + 3.0 * GELU_B * z * z)
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q * (1.0 + z * (1.0 - q))
    return torch.ones_like(z)


def _plain_product(s):
    c = s["case"]
    a = _mx_values(s["a"], c["m"])
    g = a @ _mx_values(s["gate"], c["f"]).t()
    u = a @ _mx_values(s["up"], c["f"]).t()
    out = (_act(g, c["act"]) * u).to(BF16)
    return {"out": out, "gate_up": torch.cat([g, u], 1).to(BF16)} if c["keep"] else {"out": out}


def _plain_gate_forward(s):
    f = s["case"]["f"]
    g, u = s["gate_up"][:, :f].to(F32), s["gate_up"][:, f:].to(F32)
    return _copies(_act(g, s["case"]["act"]) * u, s)


def _plain_gate_backward(s):
    f, act = s["case"]["f"], s["case"]["act"]
    g, u, dh = s["gate_up"][:, :f].to(F32), s["gate_up"][:, f:].to(F32), s["dh"].to(F32)
    return _copies(torch.cat([dh * u * _act_slope(g, act), dh * _act(g, act)], 1), s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "product": _exact_product, "gate": _exact_gate}[case["op"]](s)


def _exact_scales(x):
    """Powers of two [R, K/32]: 2^floor(log2 of a block's largest magnitude) / 256, at least 2^-127."""
    top = x.abs().unflatten(1, (-1, 32)).amax(2)
    low = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -200))))
    low = torch.where(low > top, low / 2, torch.where(2 * low <= top, 2 * low, low))     # log2's rounding
    return (low / 256).clamp(2.0 ** -127, 2.0 ** 127)


def _exact_copy(x):
    """Values under their scales before the rounding to E4M3, and the scales in the order of their buffer."""
    scale = _exact_scales(x)
    codes = (x / scale.repeat_interleave(32, 1)).clamp(-448, 448)
    r, kb = scale.shape
    ra, ka = -(-r // 128), -(-kb // 4)
    band = torch.full((ra * 128, ka * 4), 2.0 ** -127, dtype=F64, device=x.device)
    band[:r, :kb] = scale
    # row 32 q + l of band b, block 4 a + j  ->  byte ((b * ka + a) * 32 + l) * 16 + 4 q + j
    return codes, torch.einsum("bqlaj->balqj", band.reshape(ra, 4, 32, ka, 4)).reshape(-1)


def _exact_copies(y, s):
    out = {}
    if s["case"]["axis"] & ROW:
        out["row"], out["row_scale"] = _exact_copy(y)
    if s["case"]["axis"] & COL:
        if s.get("offsets") is not None:
            parts, at = [], s["offsets"].tolist()
            for lo, hi in zip(at, at[1:]):
                parts += [y[lo:hi], torch.zeros(-(hi - lo) % 128, y.shape[1], dtype=F64, device=y.device)]
            y = torch.cat(parts)
        out["col"], out["col_scale"] = _exact_copy(y.t())
    return out


def _exact_norm(s):
    c, w = s["case"], s["weight"].to(F64)
    if c["dir"] == "fwd":
        v = s["residual"].to(F64) + s["x"].to(F64)
        r = (torch.einsum("rc,rc->r", v, v) / c["cols"] + EPS).rsqrt()
        y = torch.einsum("rc,r,c->rc", v, r, w)
        out = {"sum": v, "rstd": r, **_exact_copies(y, s)}
        return {**out, "y": y} if c["keep"] else out
    # y = w * h, h = sum * rstd, of the statistic that the forward pass left
    r = s["rstd"].to(F64)
    h = s["sum"].to(F64) * r[:, None]
    dy = s["dy"].to(F64)
    along = torch.einsum("rc,c,rc->r", dy, w, h) / c["cols"]
    dx = (dy * w - h * along[:, None]) * r[:, None] + s["dsum"].to(F64)
    return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, h), **_exact_copies(dx, s)}


def _exact_act(z, act):
    """The activation and its derivative."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).to(F64)
    if act == "gelu":       # z * sigmoid(2v), v = a (z + b z^3)
        q = torch.sigmoid(2 * GELU_A * (z + GELU_B * z ** 3))
        return z * q, q + z * q * (1 - q) * 2 * GELU_A * (1 + 3 * GELU_B * z ** 2)
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    return z, torch.ones_like(z)


def _exact_product(s):
    c = s["case"]
    a, gate, up = (_mx_values(s[n], r, F64) for n, r in (("a", c["m"]), ("gate", c["f"]), ("up", c["f"])))
    g, u = torch.mm(a, gate.t()), torch.mm(a, up.t())
    out = u.mul(_exact_act(g, c["act"])[0])
    return {"out": out, "gate_up": torch.hstack([g, u])} if c["keep"] else {"out": out}


def _exact_gate(s):
    c = s["case"]
    g, u = s["gate_up"].to(F64).chunk(2, 1)
    value, slope = _exact_act(g, c["act"])
    if c["dir"] == "fwd":
        return _exact_copies(u * value, s)
    dh = s["dh"].to(F64)
    return _exact_copies(torch.hstack([slope * u * dh, value * dh]), s)
