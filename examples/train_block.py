"""Trains one pre-norm block (a dense FFN, then routed experts) on a fixed target,
entirely through the public entry points:

  forward   h = rms_norm(x);  a = gelu(h W1^T + b1);  y = a W2^T + b2 + x
            n = layer_norm(y); top-k experts of softmax(n Wr^T), their weights and
            the balance loss;  out = y + sum_k weight_k (n We[expert_k]^T)
  backward  the same calls' gradients, the products as dgrad and wgrad
  update    AdamW on the FP32 masters (32-bit states for vectors and the router,
            8-bit ones for the weight matrices), then their new MXFP8 copies

Every step is a sequence of launches on the current stream and reads nothing back;
the loss is printed from a device buffer at the end.

  python examples/train_block.py [--tokens 512] [--hidden 256] [--ffn 768] [--experts 8] [--top-k 2] [--steps 30]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp8_block_scaled_gb300 as mx  # noqa: E402


class Block:
    """Masters, their MXFP8 copies and the optimiser's states. Tokens, hidden and
    FFN sizes: multiples of 32 (the MX block)."""

    MATRICES = ("w1", "w2", "we")

    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, seed: int = 0, coef: float = 0.01):
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, device="cuda", generator=g) * shape[-1] ** -0.5

        self.top_k, self.coef = top_k, coef
        self.p = dict(w1=normal(ffn, hidden), w2=normal(hidden, ffn), we=normal(experts, hidden, hidden),
                      wr=normal(experts, hidden), b1=torch.zeros(ffn, device="cuda"), b2=torch.zeros(hidden, device="cuda"),
                      g1=torch.ones(hidden, device="cuda"), g2=torch.ones(hidden, device="cuda"),
                      c2=torch.zeros(hidden, device="cuda"))
        self.state = {k: mx.adamw_state(t, 8 if k in self.MATRICES else 32) for k, t in self.p.items()}
        self.status = mx.new_status()
        self.step_count = 0
        self.refresh()

    def refresh(self):
        """The MXFP8 copies (both orientations) of the masters."""
        self.q1 = mx.quantize(self.p["w1"], mx.MX_BOTH, status=self.status)
        self.q2 = mx.quantize(self.p["w2"], mx.MX_BOTH, status=self.status)
        self.qe = mx.quantize_stacked(self.p["we"], mx.MX_BOTH, status=self.status)

    def forward_backward(self, x, target, tokens_per_seq=None):
        """x, target: BF16 [tokens, hidden]. Returns (loss [1], balance loss [1], gradients)."""
        p, st, K = self.p, self.status, self.top_k
        T, H = x.shape

        # Dense FFN: the bias, GELU and residual in the products' epilogues.
        h, _, h_rstd = mx.layer_norm(x, p["g1"], center=False, status=st)
        h_row, h_col = mx.quantize(h, mx.MX_BOTH, status=st)
        a, z = mx.gemm_epilogue(mx.MX_FPROP, h_row, self.q1[0], bias=p["b1"], act="gelu", keep_preact=True, status=st)
        a_row, a_col = mx.quantize(a, mx.MX_BOTH, status=st)
        y, _ = mx.gemm_epilogue(mx.MX_FPROP, a_row, self.q2[0], bias=p["b2"], residual=x, status=st)

        # Routed experts: token copies ordered by expert, one product per expert.
        n, n_mean, n_rstd = mx.layer_norm(y, p["g2"], p["c2"], status=st)
        logits = n.float() @ p["wr"].T
        route = mx.router_forward(logits, K, tokens_per_seq, normalize=True, coef=self.coef, status=st)
        order = torch.argsort(route.indices.flatten(), stable=True)
        token, weight = order // K, route.weights.flatten()[order, None]
        rows = n[token]
        r_row, r_col = mx.quantize(rows, mx.MX_BOTH, group_offsets=route.group_offsets, status=st)
        e_out = mx.grouped_gemm(mx.MX_FPROP, r_row, self.qe[0], route.group_offsets, status=st)
        out = y.float().index_add(0, token, weight * e_out.float())

        diff = out - target.float()
        loss = (diff * diff).mean().view(1)
        grads = {}

        # Experts and router.
        dout = diff * (2.0 / diff.numel())
        d_rows = (weight * dout[token]).to(torch.bfloat16)
        d_weight = torch.empty(T * K, device=x.device)
        d_weight[order] = (dout[token] * e_out.float()).sum(1)
        d_row, d_col = mx.quantize(d_rows, mx.MX_BOTH, group_offsets=route.group_offsets, status=st)
        grads["we"] = mx.grouped_gemm(mx.MX_WGRAD, d_col, r_col, route.group_offsets, status=st)
        d_in = mx.grouped_gemm(mx.MX_DGRAD, d_row, self.qe[1], route.group_offsets, status=st)
        d_logits = mx.router_backward(logits, route.indices, route.load, d_weight.view(T, K), torch.ones_like(route.loss),
                                      tokens_per_seq, normalize=True, status=st)
        grads["wr"] = d_logits.T @ n.float()
        dn = (d_logits @ p["wr"]).index_add(0, token, d_in.float())
        dy, grads["g2"], grads["c2"] = mx.layer_norm_backward(dn.to(torch.bfloat16), y, p["g2"], n_mean, n_rstd, status=st)

        # Dense FFN: a layer's dgrad and wgrad in one launch.
        dy = (dy.float() + dout).to(torch.bfloat16)
        dz2, grads["b2"] = mx.epilogue_backward(dy, None, status=st)
        d2_row, d2_col = mx.quantize(dz2, mx.MX_BOTH, status=st)
        da, grads["w2"] = mx.gemm_multi([(mx.MX_DGRAD, d2_row, self.q2[1]), (mx.MX_WGRAD, d2_col, a_col)], status=st)
        dz1, grads["b1"] = mx.epilogue_backward(da, z, "gelu", status=st)
        d1_row, d1_col = mx.quantize(dz1, mx.MX_BOTH, status=st)
        dh, grads["w1"] = mx.gemm_multi([(mx.MX_DGRAD, d1_row, self.q1[1]), (mx.MX_WGRAD, d1_col, h_col)], status=st)
        _, grads["g1"], _ = mx.layer_norm_backward(dh, x, p["g1"], None, h_rstd, center=False, status=st)
        return loss, route.loss, grads

    def update(self, grads, lr: float, weight_decay: float = 0.0):
        self.step_count += 1
        for keep in (True, False):
            names = [k for k in self.p if (k in self.MATRICES) == keep]
            mx.adamw_step([self.p[k] for k in names], [grads[k] for k in names], [self.state[k] for k in names], lr,
                          weight_decay=weight_decay if keep else 0.0, step=self.step_count, seed=self.step_count,
                          status=self.status)
        self.refresh()

    def check(self):
        """Raises where a kernel reported a failure."""
        code = mx.read_status(self.status)
        if code:
            raise mx.MXError(code, "training step")


def train(tokens=512, hidden=256, ffn=768, experts=8, top_k=2, steps=30, lr=3e-3, seed=0):
    """Losses of every step (a list of floats)."""
    g = torch.Generator("cuda").manual_seed(seed + 1)
    x = torch.randn((tokens, hidden), device="cuda", generator=g).to(torch.bfloat16)
    target = torch.randn((tokens, hidden), device="cuda", generator=g).to(torch.bfloat16)
    block = Block(hidden, ffn, experts, top_k, seed)
    losses = torch.zeros(steps, device="cuda")
    for i in range(steps):
        loss, _, grads = block.forward_backward(x, target)
        losses[i] = loss[0]
        block.update(grads, lr)
    block.check()
    return losses.tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 512), ("hidden", 256), ("ffn", 768), ("experts", 8), ("top-k", 2), ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--lr", type=float, default=3e-3)
    for i, loss in enumerate(train(**vars(ap.parse_args()))):
        print(f"step {i:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
