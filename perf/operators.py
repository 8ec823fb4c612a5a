"""Measured cases of the operators around the MX products of a training step.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and through this package's entry points:

- ``adamw``: one AdamW step over many tensors at once, with its two states in
  32 or in 8 bits. It updates the FP32 masters that the weight refresh reads.
- ``layer_norm``: the layer norm (or root-mean-square norm) before a Linear,
  forward, and backward with the weight's and bias's gradients.
- ``epilogue``: the MX product with bias, activation and residual, and the
  backward pass of that epilogue (the pre-activation's gradient, which is the
  dY that dgrad and wgrad quantise, and the bias's).
- ``router``: expert choice, gate weights, per-expert counts with the grouped
  products' offsets and the balance loss; and their gradient.

A case is a dict of plain values. Both forms take what prepare() gives.
"""

import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}
STATE_BLOCK = 256                     # elements that share the scales of 8-bit states
LR, BETA1, BETA2, EPS, DECAY, STEP, SEED = 1e-3, 0.9, 0.999, 1e-8, 0.1, 100, 20260


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # Norm weights and biases of two layers: many small tensors of odd sizes in one call, latency counts.
        {"name": "adamw32 small tensors", "op": "adamw", "bits": 32, "grad": "bf16",
         "sizes": "2048,2048,10944,576,4096,64,1,33,2048,2048,10944,576,4096,64,257,1000"},
        # The dense FFN's up and down weights with FP32 gradients, states in 32 bits.
        {"name": "adamw32 dense FFN", "op": "adamw", "bits": 32, "grad": "f32", "sizes": "22413312,22413312,10944,2048"},
        # The routed experts' stacked gate_up weights [64, 2816, 2048], BF16 gradients, states in 8 bits.
        {"name": "adamw8 routed experts", "op": "adamw", "bits": 8, "grad": "bf16", "sizes": "369098752"},
        # A short batch in FP32 with an odd width and a row pitch: the smallest norm calls.
        {"name": "norm fwd small odd", "op": "layer_norm", "dir": "fwd", "rows": 33, "cols": 1009, "pad": 7, "dtype": "f32",
         "center": True},
        # The quantiser sweep's width at 16384 tokens.
        {"name": "norm fwd 16384x7168", "op": "layer_norm", "dir": "fwd", "rows": 16384, "cols": 7168, "pad": 0,
         "dtype": "bf16", "center": True},
        # The norm before the attention projections at 16384 tokens, backward with both parameter gradients.
        {"name": "norm bwd 16384x2048", "op": "layer_norm", "dir": "bwd", "rows": 16384, "cols": 2048, "pad": 0,
         "dtype": "bf16", "center": True},
        # The single Linear with bias, GELU and residual: latency counts.
        {"name": "epilogue single linear", "op": "epilogue", "dir": "fwd", "m": 256, "n": 256, "k": 512, "act": "gelu",
         "bias": True, "residual": True, "preact": False},
        # The dense FFN's up projection with bias and GELU, keeping the pre-activation for the backward pass.
        {"name": "epilogue FFN up", "op": "epilogue", "dir": "fwd", "m": 8192, "n": 10944, "k": 2048, "act": "gelu",
         "bias": True, "residual": False, "preact": True},
        # Its backward pass: dY of the activation to dY of the product, and the bias's gradient.
        {"name": "epilogue FFN up bwd", "op": "epilogue", "dir": "bwd", "m": 8192, "n": 10944, "k": 0, "act": "gelu",
         "bias": True, "residual": False, "preact": True},
        # Routing one short sequence over 64 experts, six each: latency counts.
        {"name": "router fwd 256x64", "op": "router", "dir": "fwd", "tokens": 256, "seq": 256, "experts": 64, "top_k": 6,
         "dtype": "f32", "normalize": False, "masked": 0.0},
        # Sixteen sequences of 4096 tokens, padding at places, over 64 experts.
        {"name": "router fwd 65536x64", "op": "router", "dir": "fwd", "tokens": 65536, "seq": 4096, "experts": 64, "top_k": 6,
         "dtype": "f32", "normalize": True, "masked": 0.1},
        # The backward pass with 256 experts, eight each.
        {"name": "router bwd 65536x256", "op": "router", "dir": "bwd", "tokens": 65536, "seq": 4096, "experts": 256,
         "top_k": 8, "dtype": "bf16", "normalize": True, "masked": 0.1},
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "layer_norm", "epilogue", "router"])
    if op == "adamw":
        n = _log(rng, 1, 40)
        sizes = [_log(rng, 1, 60_000_000 // n) for _ in range(n)]
        return {"op": op, "bits": rng.choice([32, 8]), "grad": rng.choice(["bf16", "f32"]), "sizes": ",".join(map(str, sizes))}
    if op == "layer_norm":
        cols = _log(rng, 1, 16384)
        rows = _log(rng, 1, min(65536, 110_000_000 // cols))
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 1, 8, 24]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "center": rng.random() < 0.75}
    if op == "epilogue":
        back = rng.random() < 0.35
        n = _log(rng, 8, 10944)
        return {"op": op, "dir": "bwd" if back else "fwd", "m": _log(rng, 1, 8192), "n": n, "k": 0 if back else 32 * _log(rng, 1, 64),
                "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": back or rng.random() < 0.75,
                "residual": (not back) and rng.random() < 0.5, "preact": back or rng.random() < 0.5}
    experts = _log(rng, 2, 512)
    tokens = _log(rng, 1, min(131072, 16_000_000 // experts))
    return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "tokens": tokens, "seq": _log(rng, max(1, tokens // 32), tokens),
            "experts": experts, "top_k": rng.randint(1, min(8, experts)), "dtype": rng.choice(["f32", "bf16"]),
            "normalize": rng.random() < 0.5, "masked": rng.choice([0.0, 0.1, 0.5])}


def work(case):
    op = case["op"]
    if op == "adamw":
        sizes = _sizes(case)
        n = sum(sizes)
        blocks = sum(-(-s // STATE_BLOCK) for s in sizes)
        states = 16 * n if case["bits"] == 32 else 4 * n + 16 * blocks
        return {"bytes": 8 * n + _size(case["grad"]) * n + states, "flops": 15 * n}
    if op == "layer_norm":
        r, c, s = case["rows"], case["cols"], _size(case["dtype"])
        stats = 8 * r if case["center"] else 4 * r
        if case["dir"] == "fwd":
            return {"bytes": 2 * r * c * s + 8 * c + stats, "flops": 8 * r * c}
        return {"bytes": 3 * r * c * s + 12 * c + stats, "flops": 14 * r * c}
    if op == "epilogue":
        m, n, k = case["m"], case["n"], case["k"]
        if case["dir"] == "fwd":
            return {"bytes": (m + n) * (k + k // 32) + 2 * m * n * (1 + case["residual"] + case["preact"]) + 4 * n * case["bias"],
                    "flops": 2 * m * n * k}
        return {"bytes": 6 * m * n + 4 * n, "flops": 12 * m * n}
    t, e, k, s = case["tokens"], case["experts"], case["top_k"], _size(case["dtype"])
    seqs = -(-t // case["seq"])
    if case["dir"] == "fwd":
        return {"bytes": t * e * s + t + 8 * t * k + 16 * e + 8 + 4 * seqs * e + 4, "flops": 8 * t * e}
    return {"bytes": 2 * t * e * s + t + 8 * t * k + 4 * seqs * e + 4, "flops": 10 * t * e}


def _size(dtype):
    return 4 if dtype == "f32" else 2


def _sizes(case):
    return [int(s) for s in case["sizes"].split(",")]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen, device=DEV, dtype=F32) * std).to(dtype)


def prepare(case, seed):
    return {"adamw": _prepare_adamw, "layer_norm": _prepare_norm, "epilogue": _prepare_epilogue, "router": _prepare_router}[case["op"]](
        case, seed)


def _prepare_adamw(case, seed):
    """Parameters, gradients and states as after some steps: moments of the
    gradients' own scale, which differs from tensor to tensor."""
    gen = _rng(seed)
    s = {"case": case, "params": [], "grads": [], "m": [], "v": [], "m_scale": [], "v_scale": [],
         "grad_scale": torch.full((1,), 0.75, device=DEV)}
    for i, n in enumerate(_sizes(case)):
        size = 10.0 ** (-2 - i % 4)
        s["params"].append(_normal(gen, n, std=0.02))
        s["grads"].append(_normal(gen, n, std=size, dtype=DTYPES[case["grad"]]))
        m = _normal(gen, n, std=0.3 * size)
        v = _normal(gen, n, std=size).square_()
        if case["bits"] == 8:
            m, ms = _encode_m(m)
            v, vs = _encode_v(v, SEED, i)
            s["m_scale"].append(ms)
            s["v_scale"].append(vs)
        s["m"].append(m)
        s["v"].append(v)
    return s


def _prepare_norm(case, seed):
    """Activations with a mean, some columns much larger than the rest."""
    gen = _rng(seed)
    r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]

    def rows(std, mean):
        x = torch.empty(r, c + case["pad"], device=DEV, dtype=dt)[:, :c]
        scale = torch.where(torch.rand(c, generator=gen, device=DEV) < 0.01, 20.0, 1.0)
        return x.copy_(_normal(gen, r, c) * (std * scale) + mean)

    s = {"case": case, "x": rows(1.0, 0.25), "weight": 1.0 + _normal(gen, c, std=0.1), "bias": _normal(gen, c, std=0.1), "eps": 1e-5}
    if case["dir"] == "bwd":
        s["dy"] = rows(0.5, 0.0)
        _, s["mean"], s["rstd"] = _plain_norm_forward({**s, "weight": None, "bias": None})
    return s


def _prepare_epilogue(case, seed):
    """Quantised activations and weights as the quantiser lays them out; a
    residual stream and a pre-activation of unit size."""
    gen = _rng(seed)
    m, n, k = case["m"], case["n"], case["k"]
    s = {"case": case, "bias": _normal(gen, n, std=0.2) if case["bias"] else None}
    if case["dir"] == "fwd":
        s["a"] = _mx_rows(_normal(gen, m, k))
        s["b"] = _mx_rows(_normal(gen, n, k, std=1.0 / math.sqrt(k)))
        s["residual"] = _normal(gen, m, n, dtype=BF16) if case["residual"] else None
    else:
        s["dy"] = _normal(gen, m, n, dtype=BF16)
        s["z"] = _normal(gen, m, n, std=1.5, dtype=BF16)
    return s


def _prepare_router(case, seed):
    """Logits with a popularity for each expert; BF16 ones hold ties."""
    gen = _rng(seed)
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = (_normal(gen, t, e) + _normal(gen, e, std=0.5)).to(DTYPES[case["dtype"]])
    mask = (torch.rand(t, generator=gen, device=DEV) >= case["masked"]).to(torch.uint8) if case["masked"] > 0 else None
    s = {"case": case, "logits": logits, "mask": mask, "coef": 0.01}
    if case["dir"] == "bwd":
        f = _plain_router_forward(s)
        s["indices"], s["load"] = f["indices"], f["load"]
        s["dweights"] = _normal(gen, t, k, std=0.1)
        s["dloss"] = torch.full((1,), 1.0, device=DEV)
    return s


# ---------------------------------------------------------------------------
# Formats in torch: MX row copies and 8-bit states
# ---------------------------------------------------------------------------

def _mx_rows(x):
    """E4M3 codes [R, K] and E8M0 scales in atoms of 128 rows x 4 blocks of 32."""
    r, k = x.shape
    blocks = x.view(r, k // 32, 32)
    exp = torch.frexp(blocks.abs().amax(2)).exponent - 1 - 8
    exp = exp.clamp(-127, 127)
    codes = (blocks * torch.exp2(-exp.to(F32))[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(r, k)
    ra, ka = -(-r // 128), -(-(k // 32) // 4)
    grid = torch.zeros(ra * 128, ka * 4, dtype=torch.uint8, device=DEV)
    grid[:r, :k // 32] = (exp + 127).to(torch.uint8)
    atoms = grid.view(ra, 4, 32, ka, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes, atoms, r, k


def _mx_values(copy, dtype=F32):
    codes, atoms, r, k = copy
    ra, ka = -(-r // 128), -(-(k // 32) // 4)
    grid = atoms.view(ra, ka, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(ra * 128, ka * 4)[:r, :k // 32]
    return (codes.view(torch.float8_e4m3fn).to(dtype).view(r, k // 32, 32) * torch.exp2(grid.to(dtype) - 127)[..., None]).view(r, k)


def _blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % STATE_BLOCK)).view(-1, STATE_BLOCK)


def _encode_m(m):
    """First moment: E4M3 with one FP32 scale for 256 elements."""
    b = _blocks(m)
    amax = b.abs().amax(1)
    tiny = amax < 2.0 ** -100
    inv = torch.where(tiny, 0.0, 448.0 / amax)
    codes = (b * inv[:, None]).to(torch.float8_e4m3fn)
    return codes.view(-1)[:m.numel()], torch.where(tiny, 0.0, amax / 448.0)


def _decode_m(codes, scale):
    return (_blocks(codes.to(F32)) * scale[:, None]).view(-1)[:codes.numel()]


def _mix(x):
    """The finaliser of MurmurHash3 for 32-bit words, held in int64."""
    x = x ^ (x >> 16)
    x = (x * 0x85EBCA6B) & 0xFFFFFFFF
    x = x ^ (x >> 13)
    x = (x * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _encode_v(v, seed, i):
    """Second moment: unsigned codes of 5 exponent and 3 mantissa bits, code 255
    the block's largest value and code 1 2**-31.75 of it, rounded up or down at
    random (so that a decay by 0.1% a step is not lost). 0 stands for 0 alone."""
    n = v.numel()
    b = _blocks(v)
    amax = b.amax(1)
    bits = (b * (1.0 / amax)[:, None]).view(torch.int32).view(-1)[:n]
    key = _mix((seed + 0x9E3779B9 * (i + 1)) & 0xFFFFFFFF)
    rand = _mix((torch.arange(n, device=v.device) + key) & 0xFFFFFFFF) & 0xFFFFF
    codes = (((bits.to(torch.int64) + rand) >> 20) - 761).clamp(1, 255)
    return torch.where(v > 0, codes, 0).to(torch.uint8), amax


def _decode_v(codes, scale):
    c = codes.to(torch.int32)
    f = torch.where(c > 0, (c + 761) << 20, 0).view(F32)
    return (_blocks(f) * scale[:, None]).view(-1)[:codes.numel()]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if case["op"] == "adamw":
        return (_own_adamw if own else _plain_adamw)(state)
    if case["op"] == "layer_norm":
        if case["dir"] == "fwd":
            y, mean, rstd = (_own_norm_forward if own else _plain_norm_forward)(state)
            return {"y": y, "mean": mean, "rstd": rstd} if case["center"] else {"y": y, "rstd": rstd}
        return (_own_norm_backward if own else _plain_norm_backward)(state)
    if case["op"] == "epilogue":
        if case["dir"] == "fwd":
            return (_own_epilogue if own else _plain_epilogue)(state)
        return (_own_epilogue_backward if own else _plain_epilogue_backward)(state)
    if case["dir"] == "fwd":
        return (_own_router_forward if own else _plain_router_forward)(state)
    return (_own_router_backward if own else _plain_router_backward)(state)


# The framework's calls ------------------------------------------------------

def _own_adamw(s):
    import mxfp8_block_scaled_gb300 as mx
    eight = s["case"]["bits"] == 8
    if eight:
        states = [mx.AdamWState(8, m, v, a, b) for m, v, a, b in zip(s["m"], s["v"], s["m_scale"], s["v_scale"])]
    else:
        states = [mx.AdamWState(32, m, v) for m, v in zip(s["m"], s["v"])]
    mx.adamw_step(s["params"], s["grads"], states, lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, step=STEP,
                  grad_scale=s["grad_scale"], seed=SEED)
    return _adamw_outputs(s)


def _own_norm_forward(s):
    import mxfp8_block_scaled_gb300 as mx
    return mx.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], center=s["case"]["center"])


def _own_norm_backward(s):
    import mxfp8_block_scaled_gb300 as mx
    dx, dw, db = mx.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], center=s["case"]["center"])
    return {"dx": dx, "dweight": dw, "dbias": db}


def _own_epilogue(s):
    import mxfp8_block_scaled_gb300 as mx
    a, b = (mx.MXTensor(c[0], c[1], c[2], c[3], mx.MX_ROWWISE) for c in (s["a"], s["b"]))
    out, z = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=s["bias"], act=s["case"]["act"], residual=s["residual"],
                              keep_preact=s["case"]["preact"])
    return {"out": out, "preact": z} if s["case"]["preact"] else {"out": out}


def _own_epilogue_backward(s):
    import mxfp8_block_scaled_gb300 as mx
    dz, dbias = mx.epilogue_backward(s["dy"], s["z"], act=s["case"]["act"])
    return {"dz": dz, "dbias": dbias}


def _own_router_forward(s):
    import mxfp8_block_scaled_gb300 as mx
    c = s["case"]
    r = mx.router_forward(s["logits"], c["top_k"], tokens_per_seq=c["seq"], token_mask=s["mask"], normalize=c["normalize"],
                          coef=s["coef"])
    return {"indices": r.indices, "weights": r.weights, "counts": r.counts, "offsets": r.group_offsets, "load": r.load, "loss": r.loss}


def _own_router_backward(s):
    import mxfp8_block_scaled_gb300 as mx
    c = s["case"]
    return {"dlogits": mx.router_backward(s["logits"], s["indices"], s["load"], s["dweights"], s["dloss"], tokens_per_seq=c["seq"],
                                          token_mask=s["mask"], normalize=c["normalize"])}


# The plain forms ------------------------------------------------------------

def _adamw_outputs(s):
    names = ("params", "m", "v", "m_scale", "v_scale")
    out = {n: s[n] for n in names if s[n]}
    if sum(map(len, out.values())) > 60:      # many tensors: one flat output of each kind
        out = {n: torch.cat([t.view(-1) for t in v]) for n, v in out.items()}
    return out


def _plain_adamw(s):
    eight = s["case"]["bits"] == 8
    p = s["params"]
    g = [x.to(F32) * s["grad_scale"] for x in s["grads"]]
    m = [_decode_m(c, a) for c, a in zip(s["m"], s["m_scale"])] if eight else s["m"]
    v = [_decode_v(c, a) for c, a in zip(s["v"], s["v_scale"])] if eight else s["v"]
    torch._foreach_mul_(m, BETA1)
    torch._foreach_add_(m, torch._foreach_mul(g, 1 - BETA1))
    torch._foreach_mul_(v, BETA2)
    sq = torch._foreach_mul(g, g)
    torch._foreach_mul_(sq, 1 - BETA2)
    torch._foreach_add_(v, sq)
    denom = torch._foreach_sqrt(v)
    torch._foreach_mul_(denom, 1 / math.sqrt(1 - BETA2 ** STEP))
    torch._foreach_add_(denom, EPS)
    update = torch._foreach_div(m, denom)
    torch._foreach_mul_(update, LR / (1 - BETA1 ** STEP))
    torch._foreach_mul_(p, 1 - LR * DECAY)
    torch._foreach_sub_(p, update)
    if eight:
        coded = [(_encode_m(x), _encode_v(y, SEED, i)) for i, (x, y) in enumerate(zip(m, v))]
        for names, k in ((("m", "m_scale"), 0), (("v", "v_scale"), 1)):
            torch._foreach_copy_(s[names[1]], [c[k][1] for c in coded])
            [to.copy_(c[k][0]) for to, c in zip(s[names[0]], coded)]
    return _adamw_outputs(s)


def _plain_norm_forward(s):
    x = s["x"].to(F32)
    mean = x.mean(1) if s["case"]["center"] else None
    d = x - mean[:, None] if s["case"]["center"] else x
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + s["eps"])
    y = d * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_backward(s):
    x, dy, rstd = s["x"].to(F32), s["dy"].to(F32), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None] if s["case"]["center"] else x) * rstd
    g = dy * s["weight"]
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if s["case"]["center"]:
        dx = dx - g.mean(1, keepdim=True)
    return {"dx": (dx * rstd).to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_epilogue(s):
    z = _mx_values(s["a"]) @ _mx_values(s["b"]).t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].to(F32)
    return {"out": y.to(BF16), "preact": z.to(BF16)} if s["case"]["preact"] else {"out": y.to(BF16)}


def _plain_epilogue_backward(s):
    dy, z, act = s["dy"].to(F32), s["z"].to(F32), s["case"]["act"]
    if act == "relu":
        dz = torch.where(z > 0, dy, 0.0)
    elif act == "gelu":
        t = torch.tanh(GELU_A * (z + GELU_B * z * z * z))
        dz = dy * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_A * (1.0 + 3.0 * GELU_B * z * z))
    elif act == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        dz = dy * (q * (1.0 + z * (1.0 - q)))
    else:
        dz = dy
    return {"dz": dz.to(BF16), "dbias": dz.sum(0)}


def _sequences(s):
    """Each token's sequence, and how many there are."""
    c = s["case"]
    return torch.arange(c["tokens"], device=DEV) // c["seq"], -(-c["tokens"] // c["seq"])


def _plain_router_forward(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    x = s["logits"].to(F32)
    valid = s["mask"].bool() if s["mask"] is not None else torch.ones(t, dtype=torch.bool, device=DEV)
    ex = torch.exp(x - x.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True) * valid[:, None]
    best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]     # ties to the lowest index
    w = torch.gather(p, 1, best)
    if c["normalize"]:
        w = w / torch.where(valid[:, None], w.sum(1, keepdim=True), 1.0)
    idx = torch.where(valid[:, None], best, -1)
    seq, seqs = _sequences(s)
    hits = torch.zeros(seqs * e + 1, dtype=torch.int64, device=DEV)
    hits.index_add_(0, torch.where(valid[:, None], seq[:, None] * e + best, seqs * e).view(-1), torch.ones(t * k, dtype=torch.int64, device=DEV))
    hits = hits[:-1].view(seqs, e)
    n = torch.zeros(seqs, device=DEV, dtype=F32).index_add_(0, seq, valid.to(F32))
    live = (n > 0).sum().clamp(min=1)
    n1 = n.clamp(min=1)[:, None]
    load = s["coef"] * e / (k * live) * hits.to(F32) / (n1 * n1)
    psum = torch.stack([q.sum(0) for q in torch.split(p, c["seq"])])
    counts = hits.sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(counts, 0)])
    return {"indices": idx.to(torch.int32), "weights": w, "counts": counts, "offsets": offsets, "load": load,
            "loss": (load * psum).sum().view(1)}


def _plain_router_backward(s):
    c = s["case"]
    x = s["logits"].to(F32)
    valid = (s["mask"].bool() if s["mask"] is not None else torch.ones(c["tokens"], dtype=torch.bool, device=DEV))[:, None]
    ex = torch.exp(x - x.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True)
    idx = s["indices"].to(torch.int64).clamp(min=0)
    dw = s["dweights"]
    if c["normalize"]:
        chosen = torch.gather(p, 1, idx)
        z = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * (chosen / z)).sum(1, keepdim=True)) / z      # exactly 0 for a single choice
    g = (s["load"] * s["dloss"])[_sequences(s)[0]].scatter_add_(1, idx, dw)
    return {"dlogits": torch.where(valid, p * (g - (p * g).sum(1, keepdim=True)), 0.0).to(s["logits"].dtype)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"adamw": _exact_adamw, "layer_norm": _exact_norm, "epilogue": _exact_epilogue, "router": _exact_router}[case["op"]](s)


def _per_element(scale, n):
    return scale.to(F64).repeat_interleave(STATE_BLOCK)[:n]


def _exact_adamw(s):
    out = {"params": [], "m": [], "v": [], "m_scale": [], "v_scale": []}
    eight = s["case"]["bits"] == 8
    for i, p in enumerate(s["params"]):
        n = p.numel()
        g = s["grads"][i].to(F64) * s["grad_scale"].to(F64)
        m, v = s["m"][i], s["v"][i]
        if eight:
            m = m.to(F64) * _per_element(s["m_scale"][i], n)
            c = v.to(F64)
            # code c >= 1: exponent field and three mantissa bits of 2**-31 (1 + j/8) ... 1
            e, j = torch.floor((c + 1) / 8) - 32, torch.remainder(c + 1, 8)
            v = torch.where(c > 0, torch.exp2(e) * (1 + j / 8), 0.0) * _per_element(s["v_scale"][i], n)
        m = BETA1 * m.to(F64) + (1 - BETA1) * g
        v = BETA2 * v.to(F64) + (1 - BETA2) * g ** 2
        hat_m, hat_v = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        out["params"].append(p.to(F64) - LR * (hat_m / (hat_v.sqrt() + EPS) + DECAY * p.to(F64)))
        if eight:
            for name, x, top in (("m_scale", m, 448.0), ("v_scale", v, 1.0)):
                out[name].append(torch.stack([q.abs().max() for q in torch.split(x, STATE_BLOCK)]) / top if n < 1_000_000 else
                                 torch.nn.functional.pad(x, (0, -n % STATE_BLOCK)).view(-1, STATE_BLOCK).abs().amax(1) / top)
            out["m"].append(None)     # codes: rounded at random or at a border
            out["v"].append(None)
        else:
            out["m"].append(m)
            out["v"].append(v)
    out = {k: v for k, v in out.items() if v}
    if sum(map(len, out.values())) > 60:
        out = {k: None if v[0] is None else torch.cat(v) for k, v in out.items()}
    return out


def _exact_norm(s):
    c = s["case"]
    x = s["x"].to(F64)
    if c["dir"] == "fwd":
        mu = x.sum(1, keepdim=True) / c["cols"] if c["center"] else torch.zeros(c["rows"], 1, device=DEV, dtype=F64)
        r = ((x - mu) ** 2).sum(1, keepdim=True).div(c["cols"]).add(s["eps"]).rsqrt()
        out = {"y": (x - mu) * r * s["weight"].to(F64) + s["bias"].to(F64), "rstd": r.view(-1)}
        return {**out, "mean": mu.view(-1)} if c["center"] else out
    # y = weight * h + bias; h = (x - mean) * rstd, of the statistics that the forward pass left
    r = s["rstd"].to(F64).view(-1, 1)
    h = (x - s["mean"].to(F64).view(-1, 1)) * r if c["center"] else x * r
    dy = s["dy"].to(F64)
    dh = dy * s["weight"].to(F64).view(1, -1)
    along = torch.einsum("rc,rc->r", dh, h).view(-1, 1) / c["cols"]
    shift = dh.sum(1, keepdim=True) / c["cols"] if c["center"] else 0.0
    return {"dx": r * (dh - shift - h * along), "dweight": torch.einsum("rc,rc->c", dy, h), "dbias": dy.sum(0)}


def _exact_act(z, act):
    """The activation and its derivative."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).to(F64)
    if act == "gelu":       # z * sigmoid(2u), u = a (z + b z^3)
        u = GELU_A * (z + GELU_B * z ** 3)
        q = torch.sigmoid(2 * u)
        return z * q, q + z * q * (1 - q) * 2 * GELU_A * (1 + 3 * GELU_B * z ** 2)
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    return z, torch.ones_like(z)


def _exact_epilogue(s):
    c = s["case"]
    if c["dir"] == "bwd":
        dz = s["dy"].to(F64) * _exact_act(s["z"].to(F64), c["act"])[1]
        return {"dz": dz, "dbias": dz.sum(0)}
    z = torch.mm(_mx_values(s["a"], F64), _mx_values(s["b"], F64).t())
    if s["bias"] is not None:
        z += s["bias"].to(F64)
    y = _exact_act(z, c["act"])[0]
    if s["residual"] is not None:
        y = y + s["residual"].to(F64)
    return {"out": y, "preact": z} if c["preact"] else {"out": y}


def _exact_router(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    x = s["logits"].to(F64)
    keep = torch.ones(t, dtype=F64, device=DEV) if s["mask"] is None else s["mask"].to(F64)
    p = torch.softmax(x, 1)
    if c["dir"] == "fwd":
        order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
        chosen = torch.zeros(t, e, dtype=F64, device=DEV).scatter_(1, order, 1.0) * keep[:, None]
        w = p.gather(1, order) * keep[:, None]
        if c["normalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        per_seq = [(a.sum(0), b.sum(0), n.sum()) for a, b, n in
                   zip(chosen.split(c["seq"]), (p * keep[:, None]).split(c["seq"]), keep.split(c["seq"]))]
        live = max(1, sum(int(n > 0) for _, _, n in per_seq))
        load = torch.stack([s["coef"] / live * (e / (k * n)) * f / n if n > 0 else torch.zeros_like(f) for f, _, n in per_seq])
        loss = sum(((e / (k * n)) * f * (q / n)).sum() for f, q, n in per_seq if n > 0) * (s["coef"] / live)
        return {"indices": None, "weights": w, "counts": None, "offsets": None, "load": load,
                "loss": torch.as_tensor(loss, dtype=F64).view(1)}
    idx = s["indices"].to(torch.int64)
    dw = s["dweights"].to(F64) * keep[:, None]
    safe = idx.clamp(min=0)
    pc = p.gather(1, safe)
    if c["normalize"]:        # w_j = p_j / z
        z = pc.sum(1, keepdim=True)
        dw = dw / z - (dw * pc).sum(1, keepdim=True) / z ** 2
    dp = torch.zeros(t, e, dtype=F64, device=DEV).scatter_add_(1, safe, dw)
    dp += s["load"].to(F64).repeat_interleave(c["seq"], 0)[:t] * s["dloss"].to(F64)
    return {"dlogits": keep[:, None] * (p * dp - p * (p * dp).sum(1, keepdim=True))}
