"""A training step of a small decoder layer and its vocabulary head, put
together from this library's calls:

    embedding -> attn_qkv_fwd -> rope_fwd -> attention core (torch) -> attn_out
    -> gated MLP -> linear_ce_fwd
    linear_ce_bwd -> gated MLP -> attn_out -> attention core -> rope_bwd
    -> attn_qkv_bwd -> grad_norm -> adamw_step

Weights are bf16 with fp32 gradients; the moments are e4m3 numbers and the
weights are rounded at random (or fp32 moments and a master copy with
--f32).  The logits of the head are never in memory as a whole.

    python examples/train_step.py [--steps 60] [--f32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from backward_tcgen05_tma_gemms_gb300 import api  # noqa: E402

SMALL = dict(d=256, F=512, H=4, Hkv=2, dh=64, V=2000, tp=2)
NAMES = ("embed", "Wq", "Wk", "Wv", "Wo", "Wg", "Wu", "W2", "head")


def init(c, seed=0, device="cuda"):
    """bf16 weights, (in, out) layout; the embedding is V x d."""
    g = torch.Generator().manual_seed(seed)
    d, F, nq, nkv, V = c["d"], c["F"], c["H"] * c["dh"], c["Hkv"] * c["dh"], c["V"]
    shapes = ((V, d), (d, nq), (d, nkv), (d, nkv), (nq, d), (d, F), (d, F), (F, d), (d, V))
    std = (0.5,) + tuple(s[0] ** -0.5 for s in shapes[1:])
    return [(torch.randn(s, generator=g) * k).to(torch.bfloat16).to(device) for s, k in zip(shapes, std)]


def core(q, k, v):
    """Causal attention of (T, H, dh) queries over (T, Hkv, dh) keys: the part
    that is not this library's."""
    T, H, dh = q.shape
    k, v = (t.repeat_interleave(H // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("thd,shd->hts", q.float(), k.float()) * dh ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    return torch.einsum("hts,shd->thd", s.softmax(-1), v.float())


def gradients(c, w, tokens, labels, plan):
    """(loss, gradients of the weights in the order of NAMES, fp32)."""
    E, Wq, Wk, Wv, Wo, Wg, Wu, W2, head = w
    H, Hkv, dh, tp = c["H"], c["Hkv"], c["dh"], c["tp"]
    T, bf16 = tokens.numel(), torch.bfloat16
    pos = torch.arange(T, device=tokens.device)
    # forward.  The output projection and the MLP compute both directions in
    # one call; without an upstream gradient yet, only their outputs are used.
    x0 = E[tokens]
    q, k, v = api.attn_qkv_fwd(x0, Wq, Wk, Wv, H, Hkv, tp)
    api.rope_fwd(plan, q, k, pos, head_dim=dh, out=(q, k))
    heads = [t.view(T, -1, dh).requires_grad_() for t in (q, k, v)]
    with torch.enable_grad():
        ctx = core(*heads)
    C = ctx.detach().reshape(T, H * dh).to(bf16)
    none = torch.zeros_like(x0)
    x1 = (x0.float() + api.attn_out_fwd_bwd(C, Wo, none, H, tp)[0]).to(bf16)
    x2 = (x1.float() + api.glu_mlp_fwd_bwd(x1, Wg, Wu, W2, none, tp)[0]).to(bf16)
    _, loss, lse = api.linear_ce_fwd(x2, head, labels, ignore_index=-100, reduction="mean")
    # backward
    dx2, dhead = api.linear_ce_bwd(x2, head, labels, lse, ignore_index=-100, reduction="mean")
    _, dx, dWg, dWu, dW2 = api.glu_mlp_fwd_bwd(x1, Wg, Wu, W2, dx2.to(bf16), tp)
    dx1 = dx2 + dx
    _, dC, dWo = api.attn_out_fwd_bwd(C, Wo, dx1.to(bf16), H, tp, dC_dtype=torch.float32)
    dq, dk, dv = (t.contiguous() for t in torch.autograd.grad(ctx, heads, dC.view(T, H, dh)))
    api.rope_bwd(plan, dq, dk, pos, out=(dq, dk))
    dx, dWq, dWk, dWv = api.attn_qkv_bwd(x0, Wq, Wk, Wv, *(t.view(T, -1) for t in (dq, dk, dv)), H, Hkv, tp)
    dE = torch.zeros(E.shape, device=E.device, dtype=torch.float32).index_add_(0, tokens, dx1 + dx)
    return loss, [dE, dWq, dWk, dWv, dWo, dWg, dWu, dW2, dhead]


def train(steps=60, f32=False, c=SMALL, T=256, lr=3e-3, seed=0):
    """Trains on one batch of a fixed random sequence; returns the losses."""
    w = init(c, seed)
    opt = api.adamw_plan(w, torch.float32 if f32 else torch.float8_e4m3fn, master=f32)
    plan = api.rope_plan(c["dh"])
    g = torch.Generator().manual_seed(seed + 1)
    tokens = torch.randint(0, c["V"], (T,), generator=g).cuda()
    labels = torch.roll(tokens, -1)
    labels[-1] = -100  # nothing follows the last token
    losses = []
    for step in range(1, steps + 1):
        loss, grads = gradients(c, w, tokens, labels, plan)
        norm = api.grad_norm(grads, max_norm=1.0)
        api.adamw_step(opt, grads, lr=lr, step=step, beta2=0.95, weight_decay=0.01, grad_scale=norm[1:],
                       seed=None if f32 else step)
        losses.append(loss)
    return [x.item() for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--f32", action="store_true", help="fp32 moments and a master copy")
    a = ap.parse_args()
    for i, x in enumerate(train(a.steps, a.f32), 1):
        if i == 1 or i % 10 == 0:
            print(f"step {i:4d}  loss {x:.4f}")
    assert api.last_device_error() == 0
