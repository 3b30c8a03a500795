"""Product with bias, activation and residual, and its gradients, against 64
bits, element by element.

What the kernels may be off by, with S = |x| |W| (magnitudes multiplied):
  sums    the tensor cores cut each partial sum at 2^-23 of it, a step takes 16
          terms in bf16 and 32 in e4m3, and up to 8 runs of K are added: (K / 16 +
          16) 2^-23 S.  fp32 as three bf16 values: accumulators of at most 32
          steps, then rounded sums of them, and products left out below 2^-24
          S: (64 + K / 64) 2^-23 S; on the fp32 pipes up to K / 32 + 64 roundings
  bias, scales   2^-22 of z
  act     its slope is at most 1.13; evaluation: 2^-18 |z| (the exponent's
          rounding times its size, where the result is not small)
  y, z    finfo.eps / 2 of the value
  dz      rounded to the operands' type: eps / 2 of it, and 2^-18 |dy| for the slope
  db      T / 8 + 64 additions
"""
import math

import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
BF, FP, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ACTS = [None, "gelu", "gelu_tanh", "silu", "tanh"]


def half(dtype):
    return torch.finfo(dtype).eps / 2


def gen(*seed):
    s = 0
    for x in seed:
        s = s * 1009 + x
    return torch.Generator(device="cuda").manual_seed(s)


def act64(z, kind):
    if kind == "gelu":
        return torch.nn.functional.gelu(z)
    if kind == "gelu_tanh":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return {"silu": torch.nn.functional.silu, "tanh": torch.tanh, None: lambda t: t}[kind](z)


def sums(t, K, S):
    if t == FP:
        return (64 + K / 32) * 2.0 ** -23 * S
    return (K / 16 + 16) * 2.0 ** -23 * S


def pitched(t, extra, shift=0):
    if not extra:
        return t
    big = torch.full((t.shape[0], t.shape[1] + extra), 3.0, device="cuda").to(t.dtype)
    v = big[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def operands(T, K, N, t, layout, g, extra=0, shift=0):
    x = torch.randn(T, K, device="cuda", generator=g)
    W = torch.randn(*((K, N) if layout == "in_out" else (N, K)), device="cuda", generator=g) * K ** -0.5
    if t == E8:
        xq, xs = api.quantize_e4m3(x)
        Wq, ws = api.quantize_e4m3(W)
        return xq, Wq, xs, ws, xq.double() * xs.double()[:, None], (Wq.double() * ws.double()[:, None]).t()
    x, W = pitched(x.to(t), extra, shift), pitched(W.to(t), extra, shift)
    return x, W, None, None, x.double(), (W if layout == "in_out" else W.t()).double()


def forward(T, K, N, t, layout="out_in", act=None, bias=FP, res=None, out=None, pre=False, extra=0, shift=0, in_place=False):
    g = gen(T, K, N)
    x, W, xs, ws, x64, W64 = operands(T, K, N, t, layout, g, extra, shift)
    b = None if bias is None else torch.randn(N, device="cuda", generator=g).to(bias)
    r = None if res is None else pitched(torch.randn(T, N, device="cuda", generator=g).to(res), extra, shift)
    r64 = 0 if r is None else r.double()
    out = out or (BF if t == E8 else t)
    buf = None
    if in_place:
        assert res == out
        buf = (r, torch.empty(T, N, dtype=out, device="cuda") if pre else None)
    y, z = api.linear_fwd(x, W, bias=b, residual=r, act=act, weight_layout=layout, x_scale=xs, w_scale=ws, want_pre=pre,
                          out_dtype=out, out=buf)
    assert api.last_device_error() == 0
    want_z = x64 @ W64 + (0 if b is None else b.double())
    S = x64.abs() @ W64.abs()
    ez = sums(t, K, S) + 2.0 ** -22 * (want_z.abs() + S)
    if pre:
        assert z.dtype == out and ((z.double() - want_z).abs() <= half(out) * want_z.abs() + ez).all()
    want = act64(want_z, act) + r64
    lim = half(out) * want.abs() + 1.2 * ez + (2.0 ** -18 * want_z.abs() if act else 0) + 2.0 ** -23 * (want.abs() + abs(r64))
    diff = (y.double() - want).abs()
    assert y.dtype == out and y.shape == (T, N) and (diff <= lim).all(), f"{(diff - lim).max().item():.3e} over"


TS = [1, 2, 7, 16, 17, 64, 65, 129, 256, 257, 520]


@pytest.mark.parametrize("T", TS)
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("t", [BF, FP])
def test_rows(T, layout, t):
    forward(T, 584, 136, t, layout, act="silu", res=t)
    forward(T, 64, 1032, t, layout, bias=None)


@pytest.mark.parametrize("T", TS)
def test_rows_e4m3(T):
    forward(T, 592, 136, E8, act="silu", res=BF)
    forward(T, 16, 1030, E8, bias=None)
    forward(T, 2064, 264, E8, bias=BF, res=FP, out=FP)


@pytest.mark.parametrize("K,N", [(1, 1), (8, 1), (1, 40), (3, 5), (63, 127), (64, 128), (65, 129), (72, 257), (1000, 100),
                                 (1001, 33), (4096, 24), (5000, 130)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("t", [BF, FP])
def test_odd_sizes(K, N, layout, t):
    for T in (1, 5, 40, 300):
        forward(T, K, N, t, layout, act="gelu", res=t, pre=True)


@pytest.mark.parametrize("K,N", [(16, 1), (32, 40), (128, 128), (144, 129), (1008, 100), (14336, 24)])
def test_odd_sizes_e4m3(K, N):
    for T in (1, 5, 40, 300):
        forward(T, K, N, E8, act="gelu", res=BF, pre=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias", [None, BF, FP])
@pytest.mark.parametrize("res", [None, BF, FP])
@pytest.mark.parametrize("out", [BF, FP])
def test_epilogues(act, bias, res, out):
    for T in (9, 300):
        for t in (BF, FP, E8):
            forward(T, 256, 192, t, "out_in", act, bias, res, out, pre=act is not None)


@pytest.mark.parametrize("extra,shift", [(8, 8), (8, 0), (3, 1)])
@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
def test_pitched(extra, shift, t, layout):
    for T in (3, 60, 300):
        forward(T, 136, 264, t, layout, "silu", FP, t, t, True, extra, shift)


@pytest.mark.parametrize("t", [BF, FP, E8])
def test_residual_in_place(t):
    for T in (1, 40, 300, 700):
        forward(T, 256, 520, t, "out_in", "gelu_tanh", FP, BF, BF, True, in_place=True)
        forward(T, 256, 523, t, "out_in", None, FP, FP, FP, in_place=True)


def test_columns_first():
    """X whose unit stride is along the rows, shared rows of X, and higher ranks."""
    for t in (BF, FP):
        for T in (24, 304):
            x = torch.randn(128, T, device="cuda").to(t).t()
            W = torch.randn(128, 72, device="cuda").to(t)
            y, _ = api.linear_fwd(x, W, out_dtype=FP)
            want, S = x.double() @ W.double(), x.double().abs() @ W.double().abs()
            assert ((y.double() - want).abs() <= sums(t, 128, S) + 2.0 ** -22 * S).all()
        one = torch.randn(1, 128, device="cuda").to(t).expand(6, 128)
        y, _ = api.linear_fwd(one, W)
        assert (y == y[:1]).all()
        x = torch.randn(2, 3, 128, device="cuda").to(t)
        y, z = api.linear_fwd(x, W, act="silu", want_pre=True)
        assert y.shape == z.shape == (2, 3, 72)
        assert torch.equal(y.view(6, 72), api.linear_fwd(x.view(6, 128), W, act="silu")[0])
        assert torch.equal(api.linear_fwd(x[0, 0], W)[0].view(1, 72), api.linear_fwd(x[0, :1], W)[0])


def test_few_rows_agree_with_many():
    """A row's result does not depend on which kernel its batch takes, beyond the order of its sums."""
    for t in (BF, E8):
        x, W, xs, ws, x64, W64 = operands(600, 1024, 384, t, "out_in", gen(1))
        S = x64.abs() @ W64.abs()
        many = api.linear_fwd(x, W, x_scale=xs, w_scale=ws, out_dtype=FP, weight_layout="out_in")[0].double()
        for T in (1, 33, 200, 256, 400):
            few = api.linear_fwd(x[:T], W, x_scale=None if xs is None else xs[:T], w_scale=ws, out_dtype=FP,
                                 weight_layout="out_in")[0].double()
            assert ((few - many[:T]).abs() <= 2 * sums(t, 1024, S[:T]) + 2.0 ** -21 * S[:T]).all()


def test_not_finite():
    """An infinity or a NaN stays in its row and its column."""
    for t in (BF, FP):
        for T in (3, 40, 300):
            x, W = torch.ones(T, 64, device="cuda").to(t), torch.ones(64, 72, device="cuda").to(t)
            x[1, 3], W[5, 7] = math.inf, math.nan
            y, _ = api.linear_fwd(x, W, bias=torch.zeros(72, device="cuda"))
            bad = torch.zeros(T, 72, dtype=torch.bool, device="cuda")
            bad[1] = bad[:, 7] = True
            assert torch.isfinite(y[~bad]).all() and torch.isinf(y[1, :7]).all() and torch.isnan(y[:, 7]).all()


@pytest.mark.parametrize("act", ACTS)
def test_far_from_zero(act):
    """Pre-activations up to the end of the types: the activation is z or 0, its slope 1 or 0 (tanh: 1 and 0)."""
    far = torch.tensor([1e38, 1e30, 1e20, 1e10, 300.0, 150.0, 101.0, 99.0, 60.0], device="cuda")
    far = torch.cat((far, -far)).to(BF)
    for T in (1, 40, 300):
        for t in (BF, FP):
            x = torch.zeros(T, 64, device="cuda").to(t)
            x[:, 0] = 1
            W = torch.zeros(64, 24, device="cuda").to(t)
            W[0, :18] = far.to(t)
            y, z = api.linear_fwd(x, W, act=act, want_pre=True)
            assert torch.equal(z[:, :18], far.to(t).expand(T, 18))
            want = act64(far.double(), act)
            assert ((y[:, :18].double() - want).abs() <= (half(t) + 2.0 ** -18) * want.abs() + 1e-20).all()
            if act:
                _, _, db = api.linear_bwd(x, W, torch.ones_like(z), pre=z, act=act)
                slope = (far > 0).double() if act != "tanh" else torch.zeros(18, device="cuda").double()
                assert ((db[:18].double() - T * slope).abs() <= 2.0 ** -18 * T).all()


def backward(T, K, N, t, layout="in_out", act=None, yt=None, grads=None, want=(1, 1, 1), extra=0, shift=0):
    g = gen(T, K, N, 7)
    x, W, _, _, x64, W64 = operands(T, K, N, t, layout, g, extra, shift)
    yt, grads = yt or t, grads or t
    dy = pitched(torch.randn(T, N, device="cuda", generator=g).to(yt), extra, shift)
    z = pitched((2 * torch.randn(T, N, device="cuda", generator=g)).to(t), extra, shift) if act else None
    dx, dW, db = api.linear_bwd(x, W, dy, pre=z, act=act, weight_layout=layout, want_dx=bool(want[0]),
                                want_dw=bool(want[1]), want_dbias=bool(want[2]), grad_dtype=grads)
    assert api.last_device_error() == 0
    dz = dy.double()
    if act:
        with torch.enable_grad():
            q = z.double().requires_grad_()
            slope, = torch.autograd.grad(act64(q, act).sum(), q)
        dz = dz * slope
    edz = (half(t) if act or yt != t else 0) * dz.abs() + (2.0 ** -18 * dy.double().abs() if act else 0)
    for got, a, b, terms, what in ((dx, dz, W64.t(), N, "dx"), (dW, x64.t(), dz, T, "dW")):
        if got is None:
            continue
        ref = a @ b
        S = a.abs() @ b.abs()
        e = edz @ b.abs() if what == "dx" else a.abs() @ edz
        if what == "dW" and layout == "out_in":
            got = got.t()
        lim = half(grads) * ref.abs() + sums(t, terms, S + e) + e * 1.01 + 2.0 ** -22 * S
        diff = (got.double() - ref).abs()
        assert got.dtype == grads and (diff <= lim).all(), f"{what}: {(diff - lim).max().item():.3e} over"
        if t == BF and T * K * N > 1 << 20:
            assert (got.double() - ref).norm() <= 5e-3 * ref.norm()
    if db is not None:
        ref = dz.sum(0)
        lim = half(grads) * ref.abs() + (T / 8 + 64) * 2.0 ** -24 * dz.abs().sum(0) + \
            (2.0 ** -18 * dy.double().abs().sum(0) if act else 0)
        assert ((db.double() - ref).abs() <= lim).all()


@pytest.mark.parametrize("T", [1, 5, 64, 200, 257, 700])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("t", [BF, FP])
def test_backward_rows(T, layout, t):
    backward(T, 136, 264, t, layout, "gelu_tanh")
    backward(T, 264, 136, t, layout)


@pytest.mark.parametrize("T,K,N", [(1, 1, 1), (3, 5, 7), (33, 65, 127), (100, 64, 1), (40, 1, 64), (77, 1001, 333), (300, 72, 1000),
                                   (2000, 40, 24)])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("t", [BF, FP])
def test_backward_odd_sizes(T, K, N, layout, t):
    backward(T, K, N, t, layout, "silu")
    backward(T, K, N, t, layout)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("yt", [BF, FP])
@pytest.mark.parametrize("grads", [BF, FP])
@pytest.mark.parametrize("t", [BF, FP])
def test_backward_types(act, yt, grads, t):
    backward(300, 128, 192, t, "out_in", act, yt, grads)
    backward(20, 128, 192, t, "in_out", act, yt, grads)


@pytest.mark.parametrize("want", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)])
def test_backward_some(want):
    for act in (None, "silu"):
        backward(90, 128, 192, BF, "in_out", act, want=want)
        backward(90, 128, 192, FP, "in_out", act, want=want)


@pytest.mark.parametrize("extra,shift", [(8, 8), (3, 1)])
@pytest.mark.parametrize("t", [BF, FP])
def test_backward_pitched(extra, shift, t):
    for layout in ("in_out", "out_in"):
        backward(90, 136, 264, t, layout, "gelu", extra=extra, shift=shift)
        backward(90, 136, 264, t, layout, None, extra=extra, shift=shift)


def test_backward_against_differences():
    """<dx, v> is the slope of <dy, y(x + h v)>, by central differences in 64 bits (error below 1e-8 at
    h = 1e-5), and so for W and the bias; in fp32 with the pre-activation of the forward call."""
    g = gen(3)
    x, W = torch.randn(20, 48, device="cuda", generator=g), torch.randn(48, 56, device="cuda", generator=g) * 0.2
    b, dy = torch.randn(56, device="cuda", generator=g), torch.randn(20, 56, device="cuda", generator=g)
    for act in ACTS:
        y, z = api.linear_fwd(x, W, bias=b, act=act, want_pre=True)
        got = api.linear_bwd(x, W, dy, pre=z if act else None, act=act)
        at = [x.double(), W.double(), b.double()]
        for i, grad in enumerate(got):
            v = torch.randn(grad.shape, device="cuda", generator=g).double()

            def loss(h):
                p = [q + h * v if j == i else q for j, q in enumerate(at)]
                return (dy.double() * act64(p[0] @ p[1] + p[2], act)).sum()
            slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
            assert abs((grad.double() * v).sum() - slope) <= 2.0 ** -15 * (grad.double() * v).abs().sum() + 1e-6


def test_empty():
    for t in (BF, FP):
        x, W = torch.empty(0, 64, device="cuda").to(t), torch.randn(64, 72, device="cuda").to(t)
        y, _ = api.linear_fwd(x, W)
        assert y.shape == (0, 72)
        dx, dW, db = api.linear_bwd(x, W, y)
        assert dx.shape == (0, 64) and not dW.any() and not db.any()


def test_rows_around_are_untouched():
    for t in (BF, FP):
        for T in (5, 40, 300):
            big = torch.full((T + 4, 112), 3.0, device="cuda").to(t)
            x, W = torch.randn(T, 64, device="cuda").to(t), torch.randn(64, 72, device="cuda").to(t)
            api.linear_fwd(x, W, out=(big[2:T + 2, 16:88], None))
            assert (big[:2] == 3).all() and (big[T + 2:] == 3).all() and (big[:, :16] == 3).all() and (big[:, 88:] == 3).all()
            big.fill_(3.0)
            dW = torch.full((64, 96), 3.0, device="cuda")
            api.linear_bwd(x, W, torch.randn(T, 72, device="cuda").to(t), out=(big[2:T + 2, 16:80], dW[:, 8:80], None))
            assert (big[:2] == 3).all() and (big[T + 2:] == 3).all() and (big[:, :16] == 3).all() and (big[:, 80:] == 3).all()
            assert (dW[:, :8] == 3).all() and (dW[:, 80:] == 3).all()


def test_results_do_not_change():
    x, W = torch.randn(900, 512, device="cuda").to(BF), torch.randn(512, 640, device="cuda").to(BF)
    dy, z = torch.randn(900, 640, device="cuda").to(BF), torch.randn(900, 640, device="cuda").to(BF)
    a, b = (api.linear_bwd(x, W, dy, pre=z, act="silu") for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    for T in (1, 64, 900):
        assert torch.equal(api.linear_fwd(x[:T], W)[0], api.linear_fwd(x[:T], W)[0])


def test_graph_and_streams():
    """Captured once, replayed with new inputs; and two calls at once on two streams."""
    cases = [(T, t) for T in (1, 40, 300) for t in (BF, FP)]
    sets = []
    for T, t in cases:
        x, W = torch.randn(T, 128, device="cuda").to(t), torch.randn(128, 136, device="cuda").to(t)
        y, z = (torch.zeros(T, 136, device="cuda").to(t) for _ in range(2))
        ws = torch.empty(max(1, api.linear_workspace_bytes(T, 128, 136, t, True)), dtype=torch.uint8, device="cuda")
        back = (torch.zeros_like(x), torch.zeros_like(W), torch.zeros(136, device="cuda"))
        sets.append((x, W, y, z, ws, back))

    def step():
        for x, W, y, z, ws, back in sets:
            api.linear_fwd(x, W, act="silu", workspace=ws, out=(y, z))
            api.linear_bwd(x, W, y, pre=z, act="silu", workspace=ws, out=back)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for x, W, *_ in sets:
            x.normal_()
            W.normal_()
        g.replay()
        torch.cuda.synchronize()
        for x, W, y, z, _, back in sets:
            want = api.linear_fwd(x, W, act="silu", want_pre=True)
            assert torch.equal(y, want[0]) and torch.equal(z, want[1])
            dx, dW, db = api.linear_bwd(x, W, y, pre=z, act="silu", grad_dtype=x.dtype)
            assert torch.equal(back[0], dx) and torch.equal(back[1], dW) and torch.equal(back[2].to(x.dtype), db)
    streams = [torch.cuda.Stream() for _ in sets]
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (x, W, *_) in zip(streams, sets):
            with torch.cuda.stream(s):
                outs.append((api.linear_fwd(x, W, act="silu")[0], x, W))
    torch.cuda.synchronize()
    for y, x, W in outs:
        assert torch.equal(y, api.linear_fwd(x, W, act="silu")[0])


def test_past_32_bit_offsets():
    """4.3 GB of outputs and residual: the last rows like any others."""
    T, N = (1 << 31) // 8192 + 7, 8192
    x, W = torch.zeros(T, 64, device="cuda").to(BF), torch.randn(64, N, device="cuda").to(BF)
    x[-9:] = torch.randn(9, 64, device="cuda").to(BF)
    y = torch.ones(T, N, dtype=BF, device="cuda")
    api.linear_fwd(x, W, residual=y, out=(y, None))
    want = x[-9:].double() @ W.double() + 1
    S = x[-9:].double().abs() @ W.double().abs()
    assert ((y[-9:].double() - want).abs() <= half(BF) * want.abs() + sums(BF, 64, S) + 2.0 ** -22 * (S + 1)).all()
    assert (y[:1000] == 1).all()


def test_refusals():
    x, W = torch.randn(4, 64, device="cuda"), torch.randn(64, 72, device="cuda")
    for call in (lambda: api.linear_fwd(x, W, act="relu"), lambda: api.linear_fwd(x, W, weight_layout="sideways")):
        with pytest.raises(ValueError, match="argument"):
            call()
    for call in (lambda: api.linear_fwd(x, W, weight_layout="out_in"), lambda: api.linear_fwd(x, W, bias=torch.zeros(71, device="cuda")),
                 lambda: api.linear_fwd(x, W, residual=torch.zeros(4, 64, device="cuda")), lambda: api.linear_fwd(x, W[0]),
                 lambda: api.linear_bwd(x, W, x)):
        with pytest.raises(ValueError, match="shape"):
            call()
    q, s = api.quantize_e4m3(x)
    p, t = api.quantize_e4m3(W.t().contiguous())
    for call in (lambda: api.linear_fwd(q, p, weight_layout="out_in"),                           # without scales
                 lambda: api.linear_fwd(x, W, x_scale=s, w_scale=t),                             # without codes
                 lambda: api.linear_fwd(q, p.t(), x_scale=s, w_scale=t),                         # (in, out) codes
                 lambda: api.linear_fwd(q[:, :50], p[:, :50], x_scale=s, w_scale=t, weight_layout="out_in",
                                        out=(torch.empty(4, 72, device="cuda").t(), None)),      # columns
                 lambda: api.linear_fwd(q[:, 8:24], p[:, 8:24], x_scale=s, w_scale=t, weight_layout="out_in"),  # off 16 bytes
                 lambda: api.linear_bwd(x, W, torch.zeros(4, 72, device="cuda"), act="silu"),    # without z
                 lambda: api.linear_fwd(x.to(BF), W),
                 lambda: api.linear_bwd(x, W, torch.zeros(4, 72, device="cuda"),
                                        workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(api.TpsError):
            call()
    with pytest.raises(ValueError, match="no CPU path"):
        api.linear_fwd(x, W, workspace=torch.empty(1 << 20, dtype=torch.uint8))
