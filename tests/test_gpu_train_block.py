"""The example block: its gradients against automatic differentiation in FP32, and
that training lowers the loss.

Tolerance of the gradients. An E4M3 operand is off by at most 2**-4 of an element
(half a unit in the last of three fraction bits), 2**-4 / sqrt(3) in the root mean
square. A gradient here depends on at most ten such operands (forward and
backward), independent of one another: sqrt(10) 2**-4 / sqrt(3) = 0.11 of its norm,
taken at twice that for the differences that the softmax and the norm form.
All experts are chosen, so that no choice depends on a rounding.
"""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from examples import train_block

pytestmark = pytest.mark.gpu


def reference(block, x, target):
    p = {k: v.detach().clone().requires_grad_() for k, v in block.p.items()}
    F, H = torch.nn.functional, x.shape[1]
    x, target = x.float(), target.float()
    h = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * p["g1"]
    y = F.gelu(h @ p["w1"].T + p["b1"], approximate="tanh") @ p["w2"].T + p["b2"] + x
    n = F.layer_norm(y, (H,), p["g2"], p["c2"])
    logits = n @ p["wr"].T
    prob = torch.softmax(logits, 1)
    out = y + torch.einsum("te,teh->th", prob, torch.einsum("th,eoh->teo", n, p["we"]))
    loss = ((out - target) ** 2).mean()
    E = prob.shape[1]
    balance = block.coef * (E / E) * prob.mean(0).sum()      # every expert chosen by every token
    (loss + balance).backward()
    return loss.detach(), balance.detach(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("tokens,hidden,ffn", [(256, 128, 384), (96, 64, 160)])
def test_gradients(tokens, hidden, ffn):
    g = torch.Generator("cuda").manual_seed(5)
    x, t = (torch.randn((tokens, hidden), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    block = train_block.Block(hidden, ffn, experts=4, top_k=4, seed=3)
    loss, balance, grads = block.forward_backward(x, t)
    block.check()
    want, want_balance, ref = reference(block, x, t)
    assert abs(float(loss) / float(want) - 1) < 0.05 and abs(float(balance) / float(want_balance) - 1) < 1e-3
    assert set(grads) == set(ref)
    off = {k: float((grads[k].float() - ref[k]).norm() / ref[k].norm()) for k in ref}
    assert all(v < 0.22 for v in off.values()), off


def test_training_lowers_the_loss():
    losses = train_block.train(tokens=256, hidden=128, ffn=384, experts=8, top_k=2, steps=30)
    assert all(l == l for l in losses) and losses[-1] < 0.9 * losses[0], losses
