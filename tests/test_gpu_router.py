"""The router's choice, weights, counts, offsets and balance loss, and their
gradient, against the float64 oracle. Whole numbers are equal.

Tolerances (u = 2**-24). p = exp(x - m) / sum: the fast exponential's argument
is rounded at |x - m| log2(e), so p is off by (|x - m| + 8) 2**-22 of itself (the
sum and the quotient included). Normalised weights are quotients of two such.
Sums of p are chains of at most 200 additions, loads five roundings. A gradient
p (g - dot) inherits p's error twice and its sums'.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, E, seed, dtype=torch.float32, pad=0, offset=0, std=1.0):
    r = workloads.philox(seed)
    x = r.standard_normal((T, E)) * std + 0.5 * r.standard_normal(E)
    buf = torch.full((T * (E + pad) + offset,), float("nan"), dtype=dtype, device="cuda")
    t = buf[offset:].view(T, E + pad)[:, :E]
    t.copy_(torch.from_numpy(x.astype(np.float32)))
    return t


def p_tol(x, f):
    with np.errstate(invalid="ignore"):
        m = np.where(f["valid"][:, None], x, 0).max(1, keepdims=True)
        d = np.where(np.isfinite(x) & f["valid"][:, None], m - x, 0.0)
    return f["p"] * (d + 8) * 2.0 ** -22 + 1e-38


def check_forward(r, x, top_k, seq, mask, normalize, coef):
    fx = f64(x)
    f = so.router(fx, top_k, seq, mask, normalize, coef)
    T, E = fx.shape
    assert np.array_equal(r.indices.cpu().numpy(), f["indices"])
    assert np.array_equal(r.counts.cpu().numpy(), f["counts"]) and np.array_equal(r.group_offsets.cpu().numpy(), f["offsets"])
    pt = p_tol(fx, f)
    rel = np.divide(pt, f["p"], out=np.zeros_like(pt), where=f["p"] > 0).clip(max=1)
    safe = np.maximum(f["indices"], 0)
    wt = np.take_along_axis(rel, safe, 1) * (f["indices"] >= 0)
    if normalize:
        wt = wt + wt.max(1, keepdims=True) + 40 * U
    assert (np.abs(f64(r.weights) - f["weights"]) <= wt * f["weights"] + 2 * U * f["weights"]).all()
    assert (np.abs(f64(r.load) - f["load"]) <= 8 * U * np.abs(f["load"])).all()
    seqs = f["load"].shape[0]
    st = np.array([pt[s * seq:(s + 1) * seq].sum(0) for s in range(seqs)]).reshape(seqs, E)
    tol = (np.abs(f["load"]) * (st + 220 * U * f["psum"])).sum() + 600 * U * abs(f["loss"])
    assert abs(float(r.loss) - f["loss"]) <= tol, (float(r.loss), f["loss"], tol)
    return f


def check_backward(dx, x, f, idx, load, dw, dloss, seq, mask, normalize):
    fx, fl = f64(x), f64(load)
    fd = f64(dw) if dw is not None else None
    ref = so.router_backward(fx, idx, fl, fd, dloss, seq, mask, normalize)
    T, E = fx.shape
    pt, p = p_tol(fx, f), f["p"]
    base = np.abs(dloss * fl[np.arange(T) // seq])
    g_abs, g_err = base.copy(), 4 * U * base
    if fd is not None:
        for t in range(T):
            if not f["valid"][t]:
                continue
            on = idx[t] >= 0
            sel, d = idx[t][on], np.abs(fd[t][on])
            e = 2 * U * d
            if normalize:
                z = p[t, sel].sum()
                spread = d + d.max()                       # every dw is taken against the first
                rel = (pt[t, sel] / np.maximum(p[t, sel], 1e-300)).clip(max=1).max() * 3 + 60 * U
                d = (spread + spread.max()) / z
                e = d * rel
            g_abs[t, sel] += d
            g_err[t, sel] += e
    dot_err = (pt * g_abs + p * g_err + 60 * U * p * g_abs).sum(1, keepdims=True)
    dot_abs = (p * g_abs).sum(1, keepdims=True)
    tol = pt * (g_abs + dot_abs) + p * (g_err + dot_err + 4 * U * (g_abs + dot_abs)) + 1e-38
    if dx.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    else:
        tol = tol + U * np.abs(ref)
    bad = ~(np.abs(f64(dx) - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.abs(f64(dx) - ref).max())


CASES = [(1, 2, 1, 1), (5, 1, 1, 5), (7, 3, 3, 2), (33, 31, 4, 33), (200, 32, 8, 64), (300, 33, 6, 100), (257, 64, 6, 257),
         (1000, 65, 5, 333), (500, 128, 8, 250), (300, 200, 8, 300), (260, 256, 8, 128), (150, 300, 8, 150), (100, 512, 32, 100),
         (40, 8, 8, 40), (64, 512, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T,E,K,seq", CASES)
def test_forward_and_backward(T, E, K, seq, normalize, dtype):
    x = make(T, E, T + E, dtype)
    g = workloads.philox(T)
    mask = g.random(T) < 0.8
    tm = torch.from_numpy(mask).cuda()
    dw = torch.from_numpy(g.standard_normal((T, K)).astype(np.float32)).cuda()
    dloss = torch.tensor([1.7], device="cuda")
    for m, t in ((None, None), (mask, tm)):
        r = mx.router_forward(x, K, tokens_per_seq=seq, token_mask=t, normalize=normalize, coef=0.3)
        f = check_forward(r, x, K, seq, m, normalize, 0.3)
        kw = dict(tokens_per_seq=seq, token_mask=t, normalize=normalize)
        for d, l, s in ((dw, dloss, 1.7), (None, dloss, 1.7), (dw, None, 0.0)):
            dx = mx.router_backward(x, r.indices, r.load, d, l, **kw)
            check_backward(dx, x, f, f["indices"], r.load, d, np.float32(s).astype(float), seq, m, normalize)
        again = mx.router_forward(x, K, tokens_per_seq=seq, token_mask=t, normalize=normalize, coef=0.3)
        assert torch.equal(again.loss, r.loss) and torch.equal(again.weights, r.weights) and torch.equal(again.load, r.load)


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (8, 0), (5, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_pitches_and_alignment(pad, offset, dtype):
    x = make(100, 72, 3, dtype, pad, offset)
    r = mx.router_forward(x, 6, tokens_per_seq=40)
    f = check_forward(r, x, 6, 40, None, False, 1.0)
    dw = torch.randn(100, 6, device="cuda")
    dx = mx.router_backward(x, r.indices, r.load, dw, r.loss, tokens_per_seq=40)
    check_backward(dx, x, f, f["indices"], r.load, dw, float(r.loss), 40, None, False)
    out = make(100, 72, 4, dtype, pad, offset)
    mx.mx_router_backward(x.data_ptr(), x.stride(0), mx.MX_F32 if dtype == torch.float32 else mx.MX_BF16, None, 100, 40, 72, 6, 0,
                          r.indices.data_ptr(), r.load.data_ptr(), dw.data_ptr(), r.loss.data_ptr(), out.data_ptr(),
                          out.stride(0), None, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, dx)
    if pad:
        assert torch.isnan(out.as_strided((99, pad), (72 + pad, 1), out.storage_offset() + 72)).all()


def test_ties_go_to_the_lowest_expert():
    x = torch.zeros((40, 100), device="cuda")
    x[:, 60:] = -0.0
    x[1, 50] = x[1, 99] = 1.0
    r = mx.router_forward(x, 4)
    idx = r.indices.cpu().numpy()
    assert (idx[0] == [0, 1, 2, 3]).all() and (idx[1] == [50, 99, 0, 1]).all() and (idx[2:] == [0, 1, 2, 3]).all()


def test_infinities_nan_and_left_out_tokens():
    T, E, K = 64, 48, 6
    x = make(T, E, 9)
    x[3] = -float("inf")                 # left out
    x[4, 4:] = -float("inf")             # four experts for six slots
    x[5, ::2] = -float("inf")
    x[6, 7] = torch.finfo(torch.float32).min              # the type's lowest value: p = 0, chosen last
    x[7] = torch.finfo(torch.float32).min
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[10:14] = False
    x[10] = float("nan")                 # garbage in masked places
    x[11] = float("inf")
    x[12, 5] = float("nan")
    r = mx.router_forward(x, K, tokens_per_seq=16, token_mask=mask, normalize=True, coef=0.5)
    f = check_forward(r, x, K, 16, mask.cpu().numpy(), True, 0.5)
    assert (f["indices"][3] == -1).all() and (f["indices"][4, 4:] == -1).all() and torch.isfinite(r.loss).all()
    dw = torch.randn(T, K, device="cuda")
    dw[10:14] = float("nan")
    dw[4, 4:] = float("nan")             # gradients of empty slots are not read into the result
    dx = mx.router_backward(x, r.indices, r.load, dw, r.loss, tokens_per_seq=16, token_mask=mask, normalize=True)
    clean = dw.clone()
    clean[10:14] = 0
    clean[4, 4:] = 0
    fx = x.clone()
    fx[10:14] = 0
    check_backward(dx, fx, so.router(f64(fx), K, 16, mask.cpu().numpy(), True, 0.5), f["indices"], r.load, clean,
                   float(r.loss), 16, mask.cpu().numpy(), True)
    assert (dx[3] == 0).all() and (dx[10:14] == 0).all() and (dx[4, 4:] == 0).all()


def test_a_nan_logit_shows_and_is_not_chosen():
    x = make(32, 40, 10)
    x[5, 3] = float("nan")
    r = mx.router_forward(x, 4, tokens_per_seq=16)
    assert torch.isnan(r.loss).all() and torch.isnan(r.weights[5]).all() and torch.isfinite(r.weights[[4, 6]]).all()
    assert not (r.indices[5] == 3).any() and int(r.counts.sum()) == 32 * 4
    dx = mx.router_backward(x, r.indices, r.load, torch.randn(32, 4, device="cuda"), torch.ones(1, device="cuda"), tokens_per_seq=16)
    assert torch.isnan(dx[5]).all() and torch.isfinite(dx[[4, 6]]).all()


def test_empty_and_fully_masked():
    r = mx.router_forward(torch.empty((0, 16), device="cuda"), 2)
    assert float(r.loss) == 0 and (r.counts == 0).all() and (r.group_offsets == 0).all() and r.indices.shape == (0, 2)
    assert mx.router_backward(torch.empty((0, 16), device="cuda"), r.indices, r.load).shape == (0, 16)
    x = make(50, 16, 11)
    none = torch.zeros(50, dtype=torch.bool, device="cuda")
    r = mx.router_forward(x, 2, tokens_per_seq=20, token_mask=none)
    assert float(r.loss) == 0 and (r.counts == 0).all() and (r.indices == -1).all() and (r.load == 0).all() and (r.weights == 0).all()
    dx = mx.router_backward(x, r.indices, r.load, torch.randn(50, 2, device="cuda"), torch.ones(1, device="cuda"), tokens_per_seq=20,
                            token_mask=none)
    assert (dx == 0).all()
    one = none.clone()
    one[45] = True                       # two of three sequences are empty
    check_forward(mx.router_forward(x, 2, tokens_per_seq=20, token_mask=one, coef=2.0), x, 2, 20, one.cpu().numpy(), False, 2.0)


def test_large_logits():
    x = make(64, 64, 12, std=200.0)
    r = mx.router_forward(x, 6, normalize=True)
    assert torch.isfinite(r.weights).all() and torch.isfinite(r.loss).all()
    assert (r.weights.sum(1) - 1).abs().max() < 1e-5


def test_many_tokens():
    """Sums over many CTAs: the loss against the float64 sums of the GPU's own p."""
    T, E, K, seq = 65536, 64, 6, 4096
    x = make(T, E, 13)
    r = mx.router_forward(x, K, tokens_per_seq=seq, coef=0.01)
    p = torch.softmax(x.double(), 1)
    want = (r.load.double() * p.view(16, seq, E).sum(1)).sum()
    assert abs(float(r.loss) / float(want) - 1) < 1e-5
    best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(r.indices.long(), best) and int(r.group_offsets[-1]) == T * K
    assert torch.equal(r.counts, torch.bincount(best.flatten(), minlength=E))
    one = mx.router_forward(x, K, coef=0.01)          # a single sequence
    assert abs(float(one.loss) / float((one.load.double() * p.sum(0)).sum()) - 1) < 1e-5 and torch.equal(one.counts, r.counts)


def test_gradient_against_differences_of_the_forward_pass():
    """Directional differences of sum(weights dw) + sum(load sum p) in FP32: off by
    h^2 of third derivatives (order 1) and 2**-22 roundings over h."""
    x = make(128, 40, 14)
    for normalize in (False, True):
        dw = torch.randn(128, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        f = mx.router_forward(x, 4, tokens_per_seq=64, normalize=normalize, coef=30.0)
        dx = mx.router_backward(x, f.indices, f.load, dw, torch.ones(1, device="cuda"), tokens_per_seq=64, normalize=normalize)
        v = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
        v.scatter_(1, f.indices.long(), v.gather(1, f.indices.long()).mul_(0.1))   # keeps most choices
        h = 1e-3
        def value(t):
            r = mx.router_forward(t, 4, tokens_per_seq=64, normalize=normalize, coef=30.0)
            same = (r.indices == f.indices).all(1)
            p = torch.softmax(t.double(), 1)
            return same, (r.weights.double() * dw).sum(1) + (f.load.double().repeat_interleave(64, 0) * p).sum(1)
        sa, a = value(x + h * v)
        sb, b = value(x - h * v)
        keep = sa & sb
        assert keep.float().mean() > 0.8
        num = ((a - b) / (2 * h))[keep]
        ana = (dx.double() * v).sum(1)[keep]
        assert ((num - ana).abs() <= 2e-3 + 1e-3 * ana.abs()).all(), (num - ana).abs().max()


def test_another_stream_and_a_captured_graph():
    x, dw = make(500, 64, 15), torch.randn(500, 6, device="cuda")
    def both():
        r = mx.router_forward(x, 6, tokens_per_seq=100, normalize=True)
        return [r.indices, r.weights, r.counts, r.group_offsets, r.load, r.loss,
                mx.router_backward(x, r.indices, r.load, dw, r.loss, tokens_per_seq=100, normalize=True)]
    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, cap))


def test_offsets_past_32_bits():
    T, E = 2 ** 23 + 40, 512
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    last = make(40, E, 16, torch.bfloat16)
    x[-40:] = last
    r = mx.router_forward(x, 4, tokens_per_seq=2 ** 23)
    s = mx.router_forward(last, 4)
    assert torch.equal(r.indices[-40:], s.indices) and torch.equal(r.weights[-40:], s.weights)
    assert torch.equal(r.indices[0].cpu(), torch.arange(4, dtype=torch.int32)) and int(r.group_offsets[-1]) == 4 * T
    dw = torch.zeros((T, 4), device="cuda")
    dw[-40:] = torch.randn(40, 4, device="cuda")
    dx = mx.router_backward(x, r.indices, r.load, dw, None, tokens_per_seq=2 ** 23)
    assert torch.equal(dx[-40:], mx.router_backward(last, s.indices, s.load, dw[-40:].clone(), None))
    assert (dx[:1000] == 0).all()


def test_offsets_drive_the_grouped_product():
    """counts and group_offsets as the grouped products take them."""
    T, E, K, H, N = 300, 8, 2, 64, 128
    x = make(T, E, 17)
    h = workloads.normal_bf16((T, H), 18).cuda()
    w = workloads.normal_bf16((E, N, H), 19, 0.1).cuda()
    r = mx.router_forward(x, K)
    order = torch.argsort(r.indices.flatten(), stable=True)
    rows = h[order // K].contiguous()
    a, _ = mx.quantize(rows, mx.MX_ROWWISE)
    b, _ = mx.quantize_stacked(w, mx.MX_ROWWISE)
    st = mx.new_status()
    out = mx.grouped_gemm(mx.MX_FPROP, a, b, r.group_offsets, status=st)
    assert mx.read_status(st) == 0
    e = r.indices.flatten()[order].long()
    ref = torch.einsum("rh,rnh->rn", rows.float(), w[e].float())
    assert (out.float() - ref).norm() / ref.norm() < 0.06        # two E4M3 operands: 2**-4 each at most


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K,seq", [(32, 40, 3, 1), (33, 40, 3, 1), (2000, 64, 6, 3), (500, 300, 8, 7), (4100, 512, 2, 2),
                                       (700, 5, 2, 20)])
def test_many_sequences(T, E, K, seq, dtype):
    """Around and above the number of sequences that one launch adds; the last
    sequence is shorter, and some have no valid token."""
    x = make(T, E, T + 3 * E, dtype)
    g = workloads.philox(T + 1)
    mask = (g.random(T) < 0.7) & (g.random((T + seq - 1) // seq) < 0.8).repeat(seq)[:T]
    tm = torch.from_numpy(mask).cuda()
    dw = torch.from_numpy(g.standard_normal((T, K)).astype(np.float32)).cuda()
    dloss = torch.tensor([-0.6], device="cuda")
    for m, t in ((None, None), (mask, tm)):
        r = mx.router_forward(x, K, tokens_per_seq=seq, token_mask=t, coef=0.2)
        f = check_forward(r, x, K, seq, m, False, 0.2)
        dx = mx.router_backward(x, r.indices, r.load, dw, dloss, tokens_per_seq=seq, token_mask=t)
        check_backward(dx, x, f, f["indices"], r.load, dw, np.float32(-0.6).astype(float), seq, m, False)
