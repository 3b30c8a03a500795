"""The example's training step: its gradients against torch autograd in
float64 of the same layer, and that training it works, with fp32 moments and
with e4m3 moments.

The step rounds activations and gradients to bf16 between its calls; the
whole chain is held to the framework's bf16 tolerances, loosened by the
number of roundings a gradient passes through (about eight, each 2^-8 at
most of its operand): 3e-2 in the Frobenius norm."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def turned(x, dh):
    T = x.shape[0]
    f = 10000.0 ** (-torch.arange(0, dh, 2, dtype=torch.float64, device=x.device) / dh)
    a = torch.arange(T, dtype=torch.float64, device=x.device)[:, None, None] * f
    lo, hi = x[..., :dh // 2], x[..., dh // 2:]
    return torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1)


def test_gradients_against_autograd():
    import train_step as ex
    from backward_tcgen05_tma_gemms_gb300 import api
    c, T = ex.SMALL, 192
    w = ex.init(c)
    g = torch.Generator().manual_seed(5)
    tokens, labels = (torch.randint(0, c["V"], (T,), generator=g).cuda() for _ in range(2))
    labels[10:20] = -100
    loss, grads = ex.gradients(c, w, tokens, labels, api.rope_plan(c["dh"]))
    assert api.last_device_error() == 0
    p = [t.double().requires_grad_() for t in w]
    E, Wq, Wk, Wv, Wo, Wg, Wu, W2, head = p
    x0 = E[tokens]
    q, k, v = ((x0 @ W).view(T, -1, c["dh"]) for W in (Wq, Wk, Wv))
    q, k = turned(q, c["dh"]), turned(k, c["dh"])
    k, v = (t.repeat_interleave(c["H"] // c["Hkv"], 1) for t in (k, v))
    s = torch.einsum("thd,shd->hts", q, k) * c["dh"] ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    x1 = x0 + torch.einsum("hts,shd->thd", s.softmax(-1), v).reshape(T, -1) @ Wo
    x2 = x1 + (torch.nn.functional.silu(x1 @ Wg) * (x1 @ Wu)) @ W2
    want = torch.nn.functional.cross_entropy(x2 @ head, labels, ignore_index=-100)
    want.backward()
    assert abs(loss.item() - want.item()) <= 2e-2 * want.item()
    for name, a, b in zip(ex.NAMES, grads, p):
        assert (a.double() - b.grad).norm() <= 3e-2 * b.grad.norm(), name


@pytest.mark.parametrize("f32", [True, False])
def test_training_lowers_the_loss(f32):
    import train_step as ex
    from backward_tcgen05_tma_gemms_gb300 import api
    losses = ex.train(steps=40, f32=f32)
    assert api.last_device_error() == 0
    assert losses[-1] < 0.25 * losses[0], losses[::8]
