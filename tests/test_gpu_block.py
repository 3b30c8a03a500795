"""The operators between the products as a layer uses them together: a norm in
front of a biased two-product MLP whose branch goes through dropout into the
residual stream, and the next norm -- forward and backward, against autograd
in 64 bits with the same mask; and one token of it on e4m3 numbers.

Between the calls activations and gradients are bf16: a gradient passes
through about eight such roundings, each at most 2^-8 of its operand, which
bounds the whole chain at 3e-2 in the Frobenius norm; in fp32 the same chain
is held to 1e-5."""
import pytest
import torch

import philox_plain
from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
P, SEED, SITE = 0.2, 77, 3


def weights(t, d=128, F=320, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)
    return [x.to(t) for x in (1 + 0.2 * r(d), r(d, F) * d ** -0.5, r(F) * 0.3, r(F, d) * F ** -0.5, r(d) * 0.3, 1 + 0.2 * r(d))]


def step(x, res, w, dy, dh):
    """Outputs and gradients through the library's calls."""
    n1, W1, b1, W2, b2, n2 = w
    y1, _, h1, r1 = api.rmsnorm_fwd(x, n1, residual=res)
    a, z = api.linear_fwd(y1, W1, bias=b1, act="gelu_tanh", want_pre=True)
    m, _ = api.linear_fwd(a, W2, bias=b2)
    y2, _, h2, r2 = api.rmsnorm_fwd(m, n2, residual=h1, dropout=P, seed=SEED, site=SITE)
    t = x.dtype
    dm, dh1, dn2 = api.rmsnorm_bwd(dy, h2, n2, r2, dh=dh, dropout=P, seed=SEED, site=SITE)
    da, dW2, db2 = api.linear_bwd(a, W2, dm)
    dy1, dW1, db1 = api.linear_bwd(y1, W1, da.to(t), pre=z, act="gelu_tanh")
    dx, dres, dn1 = api.rmsnorm_bwd(dy1.to(t), h1, n1, r1, dh=dh1)
    assert dx is dres
    return [y2, h2, dx, dn1, dW1, db1, dW2, db2, dn2]


def reference(x, res, w, dy, dh):
    p = [t.double().requires_grad_() for t in (x, *w)]
    xx, n1, W1, b1, W2, b2, n2 = p
    mask = torch.from_numpy(philox_plain.mask(tuple(x.shape), P, SEED, SITE)).cuda()

    def norm(v, n):
        return v * n / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    h1 = xx + res.double()
    a = torch.nn.functional.gelu(norm(h1, n1) @ W1 + b1, approximate="tanh")
    h2 = h1 + (a @ W2 + b2) * mask
    y2 = norm(h2, n2)
    ((y2 * dy.double()).sum() + (h2 * dh.double()).sum()).backward()
    return [y2.detach(), h2.detach(), *(q.grad for q in p)]


@pytest.mark.parametrize("T", [1, 37, 300])
@pytest.mark.parametrize("t,tol", [(BF, 3e-2), (FP, 1e-5)])
def test_forward_and_gradients(T, t, tol):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, res, dy, dh = (torch.randn(T, 128, device="cuda", generator=g).to(t) for _ in range(4))
    w = weights(t)
    got, want = step(x, res, w, dy, dh), reference(x, res, w, dy, dh)
    assert api.last_device_error() == 0
    for name, a, b in zip(("y2", "h2", "dx", "dn1", "dW1", "db1", "dW2", "db2", "dn2"), got, want):
        assert a.shape == b.shape and (a.double() - b).norm() <= tol * b.norm(), name


def test_beside_an_eager_graph():
    """The backward calls captured into a CUDA graph while an eager autograd graph of the same leaves lives."""
    w = [p.requires_grad_() for p in weights(BF)]
    x, res, dy, dh = (torch.randn(16, 128, device="cuda").to(BF) for _ in range(4))
    x.requires_grad_()
    eager = (x.float() @ w[1].float()).sum()
    plain = [p.detach() for p in w]
    want = step(x.detach(), res, plain, dy, dh)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(x.detach(), res, plain, dy, dh)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    eager.backward()
    assert x.grad is not None and w[1].grad is not None


def test_one_token_on_e4m3():
    """Norm with an e4m3 output into products of e4m3 weights, back into the residual stream in place.  An
    e4m3 number is off by 2^-4 at most, evenly over a step: 2^-4 / sqrt(3) in the norm, and 2^-10 of the
    row's scale below its normal numbers; each product has two such factors, and there are two products:
    2 sqrt(2) 2^-4 / sqrt(3) < 0.11."""
    n1, W1, b1, W2, b2, _ = weights(BF, 256, 640)
    q1, s1 = api.quantize_e4m3(W1.t().contiguous())
    q2, s2 = api.quantize_e4m3(W2.t().contiguous())
    for T in (1, 5, 200):
        stream, x = (torch.randn(T, 256, device="cuda").to(BF) for _ in range(2))
        before = stream.clone()
        y, ys, h, rstd = api.rmsnorm_fwd(x, n1, residual=stream, out_dtype=torch.float8_e4m3fn)
        a, _ = api.linear_fwd(y, q1, bias=b1, act="silu", x_scale=ys, w_scale=s1, weight_layout="out_in")
        aq, as_ = api.quantize_e4m3(a)
        api.linear_fwd(aq, q2, bias=b2, residual=h, x_scale=as_, w_scale=s2, weight_layout="out_in", out=(h, None))
        total = x.double() + before.double()
        want = total * n1.double() / torch.sqrt(total.square().mean(1, keepdim=True) + 1e-6)
        want = torch.nn.functional.silu(want @ W1.double() + b1.double()) @ W2.double() + b2.double()
        assert ((h.double() - total) - want).norm() <= 0.11 * want.norm() + 2 * 2.0 ** -8 * total.norm()
        assert torch.equal(stream, before)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T", [1, 8, 64, 300])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_products_right_behind_what_they_read(kind, T, captured):
    """A few-row product is started before the kernel in front of it ends: in a chain through the same
    buffers, every call sees the rows and weights of the call before, as with a wait after each."""
    g = torch.Generator(device="cuda").manual_seed(T)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    xs = [torch.randn(T, 512, device="cuda", generator=g).to(t) for _ in range(6)]
    ws = [(torch.randn(512, 512, device="cuda", generator=g) / 20).to(t) for _ in range(6)]
    h, r, y, W = torch.empty_like(xs[0]), torch.empty(T, device="cuda"), torch.empty_like(xs[0]), torch.empty_like(ws[0])
    q = (torch.empty(T, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, device="cuda"))
    qw = (torch.empty(512, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(512, device="cuda"))

    def chain(wait):
        out = []
        for x, w in zip(xs, ws):
            for weights_last in (False, True):
                if kind == "e4m3":
                    pair = [lambda: api.quantize_e4m3(y if weights_last else x, out=q), lambda: api.quantize_e4m3(w, out=qw)]
                else:
                    pair = [lambda: api.rmsnorm_fwd(y if weights_last else x, out=(h, None, None, r)),
                            lambda: api.rmsnorm_fwd(w, out=(W, None, None, torch.empty(512, device="cuda")))]
                for f in pair if weights_last else pair[::-1]:
                    f()
                    wait()
                if kind == "e4m3":
                    api.linear_fwd(q[0], qw[0], x_scale=q[1], w_scale=qw[1], weight_layout="out_in", out=(y, None))
                else:
                    api.linear_fwd(h, W, weight_layout="out_in", out=(y, None))
                wait()
                out.append(y.clone())
        return out
    want = chain(torch.cuda.synchronize)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(lambda: None)
        graph.replay()
    else:
        got = chain(lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
