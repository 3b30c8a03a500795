"""Residual addition and root-mean-square norm against their formulas in 64
bits, element by element.

What an fp32 kernel may be off by (u = 2^-24, one rounding), beside the output's
own rounding (finfo.eps / 2 of the value):
  h     the dropped value's product and the addition, one u each, and where h is
        bf16 a value next to the middle of two may fall on the other side:
        eps / 2 + 2 u of |x| scale + |res|
  rstd  a sum of d squares in at most 64 + 16 + 5 + 16 steps a number (a thread's, the warps'
        joins), the mean, the root and the reciprocal: under 64 u in the root
  y     rstd's 64 u and two products
  codes half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its
        normal numbers
  dsum  r (g - n mean) + dh: 8 u of each term's magnitude, and the mean's own sum
        of d products in up to 128 steps: 128 u of mean |g n|
  dw    a sum over rows in steps: rows a block, blocks / 8, 16 more, each one u
        of the sum of magnitudes
"""
import math

import numpy as np
import pytest
import torch

import philox_plain
from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pitched(t, extra, shift=0):
    """The same values as rows of a wider buffer."""
    if extra == 0:
        return t
    big = torch.full((t.shape[0], t.shape[1] + extra), 7.0, device="cuda").to(t.dtype)
    v = big[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def mask64(shape, p, seed, site):
    return torch.from_numpy(philox_plain.mask(shape, p, seed, site)).cuda() if p else torch.ones(shape, device="cuda").double()


def forward(T, d, xt, rt=None, wt=FP, out=None, p=0.0, seed=11, site=2, extra=0, shift=0, eps=1e-6, in_place=False):
    g = gen(T * 1000 + d)
    x = pitched((torch.randn(T, d, device="cuda", generator=g) * 3).to(xt), extra, shift)
    res = None if rt is None else pitched(torch.randn(T, d, device="cuda", generator=g).to(rt), extra, shift)
    w = None if wt is None else (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(wt)
    x64, r64 = x.double(), None if res is None else res.double()
    kw = dict(residual=res, eps=eps, dropout=p, seed=seed, site=site, out_dtype=out)
    if in_place:
        y = torch.empty(T, d, dtype=out or xt, device="cuda")
        y, scale, h, rstd = api.rmsnorm_fwd(x, w, out=(y, None, res, torch.empty(T, device="cuda")), **kw)
        assert h.data_ptr() == res.data_ptr()
    else:
        y, scale, h, rstd = api.rmsnorm_fwd(x, w, **kw)
    total = x64 * mask64((T, d), p, seed, site)
    if r64 is not None:
        total = total + r64
    if res is None and p == 0.0:
        assert h is None
        got = total
    else:
        assert h.dtype == (xt if rt is None else rt)
        lim = (half(h.dtype) + 2 * U) * total.abs() + 2 * U * (x64.abs() * 2 + (0 if r64 is None else r64.abs()))
        assert ((h.double() - total).abs() <= lim).all()
        got = h.double()
    root = torch.sqrt(got.square().mean(1) + eps)
    assert ((rstd.double() * root - 1).abs() <= 64 * U).all()
    u = got * (1.0 if w is None else w.double())
    want = u / root[:, None]
    if out == torch.float8_e4m3fn:
        top = u.abs().amax(1, keepdim=True)
        assert ((scale.double() - (top[:, 0] / 448 / root)).abs() <= 70 * U * scale.double()).all()
        back = y.double() * scale.double()[:, None]
        lim = torch.maximum(want.abs() * 2.0 ** -4, scale.double()[:, None] * 2.0 ** -10) * (1 + 1e-3) + 80 * U * want.abs()
        assert ((back - want).abs() <= lim).all()
        assert (y.double().abs().amax(1) == 448).all()
        if u.dtype == torch.float64 and xt == BF and rt in (None, BF) and wt in (None, BF):
            # products of bf16 values are exact in fp32: so are the codes, ties to even
            q = ((u * 0.875) / (top / 512)).float().clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(q.view(torch.uint8), y.view(torch.uint8))
    else:
        assert scale is None and y.dtype == (out or xt)
        assert ((y.double() - want).abs() <= (half(y.dtype) + 70 * U) * want.abs()).all()


SIZES = [(1, 1), (1, 8), (3, 5), (2, 64), (9, 264), (300, 96), (5, 1111), (17, 4096), (2, 4104), (3, 8200), (2, 16384),
         (2, 16392), (2, 20001), (700, 512)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("xt", [BF, FP])
def test_forward_sizes(T, d, xt):
    forward(T, d, xt, rt=xt, wt=xt)
    forward(T, d, xt, out=torch.float8_e4m3fn, wt=xt)


@pytest.mark.parametrize("xt", [BF, FP])
@pytest.mark.parametrize("rt", [None, BF, FP])
@pytest.mark.parametrize("wt", [None, BF, FP])
@pytest.mark.parametrize("out", [BF, FP, torch.float8_e4m3fn])
def test_forward_types(xt, rt, wt, out):
    for T, d in ((6, 1024), (5, 77)):
        forward(T, d, xt, rt, wt, out)


@pytest.mark.parametrize("p", [0.1, 0.5, 1.0, 1e-6])
@pytest.mark.parametrize("rt", [None, BF, FP])
@pytest.mark.parametrize("T,d", [(7, 136), (5, 77), (2, 16400)])
def test_forward_dropout(T, d, rt, p):
    if p == 1.0 and rt is None:
        return  # nothing is left: y = 0 is checked below
    forward(T, d, BF, rt, BF, p=p, seed=2 ** 63 + 5, site=2 ** 33 + 1)


def test_everything_dropped_and_zero_rows():
    x = torch.randn(4, 64, device="cuda")
    y, _, h, rstd = api.rmsnorm_fwd(x, dropout=1.0, seed=1)
    assert not y.any() and not h.any() and torch.allclose(rstd, torch.full_like(rstd, 1e3))
    z = torch.zeros(3, 64, device="cuda")
    z[1] = 1.0
    q, scale, _, _ = api.rmsnorm_fwd(z, out_dtype=torch.float8_e4m3fn)
    assert not q[0].float().any() and scale[0] == 0 and (q[1].float() == 448).all() and scale[2] == 0
    q, scale = api.quantize_e4m3(z * 1e-31)
    assert not q.float().any() and not scale.any()


@pytest.mark.parametrize("extra,shift", [(8, 8), (3, 1), (8, 0)])
def test_forward_pitched_rows(extra, shift):
    for d in (1024, 1031):
        forward(6, d, BF, BF, BF, extra=extra, shift=shift)
        forward(6, d, FP, BF, BF, out=BF, extra=extra, shift=shift)


@pytest.mark.parametrize("d", [1024, 77, 16400])
def test_residual_in_place(d):
    forward(6, d, BF, BF, BF, in_place=True)
    forward(6, d, FP, BF, BF, out=BF, p=0.25, in_place=True)


@pytest.mark.parametrize("d", [1024, 77, 20000])
def test_output_over_the_input(d):
    x = torch.randn(5, d, device="cuda")
    want = api.rmsnorm_fwd(x)[0]
    y = x.clone()
    api.rmsnorm_fwd(y, out=(y, None, None, torch.empty(5, device="cuda")))
    assert torch.equal(y, want)


def test_shapes_and_shared_residual():
    x = torch.randn(2, 3, 4, 64, device="cuda").to(BF)
    y, scale, h, rstd = api.rmsnorm_fwd(x, out_dtype=torch.float8_e4m3fn, residual=x)
    assert y.shape == x.shape and scale.shape == rstd.shape == (2, 3, 4) and h.shape == x.shape
    one = torch.randn(64, device="cuda")
    y, _, _, rstd = api.rmsnorm_fwd(one)
    assert y.shape == (64,) and rstd.numel() == 1
    rows = torch.randn(1, 64, device="cuda").expand(6, 64)  # a residual that the rows share
    x = torch.randn(6, 64, device="cuda")
    _, _, h, _ = api.rmsnorm_fwd(x, residual=rows)
    assert torch.equal(h, x + rows)
    e = torch.empty(0, 64, device="cuda")
    assert api.rmsnorm_fwd(e, residual=e)[0].shape == (0, 64)


def test_not_finite():
    """NaN and infinities stay in their rows."""
    x = torch.randn(5, 256, device="cuda")
    x[1, 3], x[3, 7] = math.nan, math.inf
    for out in (FP, torch.float8_e4m3fn):
        y, scale, _, _ = api.rmsnorm_fwd(x, out_dtype=out)
        v = y.float() if scale is None else y.float() * scale[:, None]
        assert torch.isfinite(v[[0, 2, 4]]).all() and torch.isnan(v[1]).all() and torch.isnan(v[3, 7])
    q, scale = api.quantize_e4m3(x)
    assert torch.isnan(scale[1]) and torch.isinf(scale[3]) and torch.isfinite(scale[[0, 2, 4]]).all()


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("xt", [BF, FP])
def test_quantize(T, d, xt):
    x = (torch.randn(T, d, device="cuda", generator=gen(d)) * torch.exp(4 * torch.randn(T, 1, device="cuda", generator=gen(T)))).to(xt)
    x[:, 0] += 1e-3
    q, scale = api.quantize_e4m3(x)
    top = x.double().abs().amax(1)
    assert ((scale.double() * 448 / top - 1).abs() <= 2 * U).all()
    want = (x.double() * 0.875) / (top / 512)[:, None]
    assert ((q.double() - want).abs() <= torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 4 * U)).all()
    if xt == BF:
        assert torch.equal(q.view(torch.uint8), want.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))


def backward(T, d, yt, ht, wt=FP, dh=True, p=0.0, x_dtype=None, extra=0, shift=0, seed=5, site=9):
    g = gen(T + d)
    h = pitched((torch.randn(T, d, device="cuda", generator=g) * 2).to(ht), extra, shift)
    dy = pitched(torch.randn(T, d, device="cuda", generator=g).to(yt), extra, shift)
    up = pitched(torch.randn(T, d, device="cuda", generator=g).to(ht), extra, shift) if dh else None
    w = None if wt is None else (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(wt)
    rstd = (h.float().square().mean(1) + 1e-6).rsqrt()
    dx, dres, dw = api.rmsnorm_bwd(dy, h, w, rstd, dh=up, dropout=p, seed=seed, site=site, x_dtype=x_dtype)
    r = rstd.double()[:, None]
    gg = dy.double() * (1.0 if w is None else w.double())
    n = h.double() * r
    mean = (gg * n).mean(1, keepdim=True)
    want = r * (gg - n * mean)
    mags = r * (gg.abs() + n.abs() * mean.abs())
    if dh:
        want = want + up.double()
        mags = mags + up.double().abs()
    lim = 8 * U * mags + 128 * U * r * n.abs() * (gg * n).abs().mean(1, keepdim=True)
    assert ((dres.double() - want).abs() <= half(ht) * want.abs() + lim).all()
    m = mask64((T, d), p, seed, site)
    xt = x_dtype or ht
    assert dx.dtype == xt and dres.dtype == ht
    assert ((dx.double() - want * m).abs() <= (half(xt) + U) * (want * m).abs() + lim * m).all()
    assert (dx is dres) == (p == 0.0 and xt == ht)
    steps = T / 152 + 152 * 4 / 8 + 32
    assert ((dw.double() - (dy.double() * n).sum(0)).abs() <= (steps + 4) * U * (dy.double() * n).abs().sum(0)).all()


@pytest.mark.parametrize("T,d", SIZES + [(2000, 4096), (5000, 64), (1300, 1111)])
@pytest.mark.parametrize("t", [BF, FP])
def test_backward_sizes(T, d, t):
    backward(T, d, t, t, t)


@pytest.mark.parametrize("yt", [BF, FP])
@pytest.mark.parametrize("ht", [BF, FP])
@pytest.mark.parametrize("wt", [None, BF, FP])
@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward_types(yt, ht, wt, dh, p):
    for T, d in ((40, 1024), (9, 77)):
        backward(T, d, yt, ht, wt, dh, p)
        backward(T, d, yt, ht, wt, dh, p, x_dtype=yt)


@pytest.mark.parametrize("extra,shift", [(8, 8), (3, 1)])
def test_backward_pitched_rows(extra, shift):
    backward(30, 1024, BF, BF, BF, extra=extra, shift=shift, p=0.1)
    backward(30, 16400, BF, FP, BF, extra=extra, shift=shift)


@pytest.mark.parametrize("d", [512, 77, 20000])
def test_backward_in_place(d):
    h, dy, up = (torch.randn(50, d, device="cuda") for _ in range(3))
    rstd = (h.square().mean(1) + 1e-6).rsqrt()
    want = api.rmsnorm_bwd(dy, h, None, rstd, dh=up, dropout=0.2, seed=3)
    a, b, w = dy.clone(), up.clone(), torch.empty(d, device="cuda")
    api.rmsnorm_bwd(a, h, None, rstd, dh=b, dropout=0.2, seed=3, out=(a, b, w))
    assert all(torch.equal(x, y) for x, y in zip(want, (a, b, w)))


def test_backward_outputs_left_out():
    h, dy = torch.randn(20, 64, device="cuda"), torch.randn(20, 64, device="cuda")
    rstd = (h.square().mean(1) + 1e-6).rsqrt()
    full = api.rmsnorm_bwd(dy, h, None, rstd)
    dx, dres, dw = api.rmsnorm_bwd(dy, h, None, rstd, want_dweight=False)
    assert dw is None and torch.equal(dx, full[0])
    dw = torch.zeros(64, device="cuda")
    api.rmsnorm_bwd(dy, h, None, rstd, out=(None, None, dw))
    assert torch.equal(dw, full[2])
    e = torch.empty(0, 64, device="cuda")
    dw = api.rmsnorm_bwd(e, e, None, torch.empty(0, device="cuda"))[2]
    assert not dw.any()


def test_backward_against_differences():
    """<dx, v> is the slope of <dy, y(h + t v)>, and <dw, v> that of the weight's: central differences
    of the formula in 64 bits, whose own error (t^2 / 6 times a third derivative of about 10 for rows
    of size 1, and 2^-53 / t) is below 1e-8 at t = 1e-5."""
    h, dy, v = (torch.randn(6, 48, device="cuda", generator=gen(i)) for i in range(3))
    w = 1 + 0.2 * torch.randn(48, device="cuda", generator=gen(4))
    rstd = (h.square().mean(1) + 1e-6).rsqrt()
    dx, _, dw = api.rmsnorm_bwd(dy, h, w, rstd)

    def loss(a, b):
        return (dy.double() * a * b / torch.sqrt(a.square().mean(1, keepdim=True) + 1e-6)).sum()
    t, hd, wd, vd = 1e-5, h.double(), w.double(), v.double()
    slope = (loss(hd + t * vd, wd) - loss(hd - t * vd, wd)) / (2 * t)
    assert abs((dx.double() * vd).sum() - slope) <= 200 * U * (dx.double() * vd).abs().sum() + 1e-6
    slope = (loss(hd, wd + t * vd[0]) - loss(hd, wd - t * vd[0])) / (2 * t)
    assert abs((dw.double() * vd[0]).sum() - slope) <= 200 * U * (dw.double() * vd[0]).abs().sum() + 1e-6


def test_results_do_not_change():
    x, dy = (torch.randn(3000, 1024, device="cuda").to(BF) for _ in range(2))
    w = torch.randn(1024, device="cuda")
    rstd = api.rmsnorm_fwd(x, w)[3]
    a, b = (api.rmsnorm_bwd(dy, x, w, rstd) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_workspace_and_wrong_outputs_are_refused():
    h = torch.randn(20, 64, device="cuda")
    rstd = torch.ones(20, device="cuda")
    with pytest.raises(api.TpsError) as e:
        api.rmsnorm_bwd(h, h, None, rstd, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == api.ERR_WORKSPACE
    with pytest.raises(ValueError, match="no CPU path"):
        api.rmsnorm_bwd(h, h, None, rstd, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        api.rmsnorm_fwd(h, torch.ones(63, device="cuda"))
    with pytest.raises(api.TpsError):
        api.rmsnorm_fwd(h.t())


def test_past_32_bit_offsets():
    """4.3 GB of rows: the last ones, and their mask, like any others."""
    T, d = (1 << 31) // 4096 + 5, 4096
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    x[-3:] = torch.randn(3, d, device="cuda").to(BF)
    rstd = torch.empty(T, device="cuda")
    api.rmsnorm_fwd(x, out=(x, None, None, rstd), eps=1e-6)
    assert ((x[-3:].double().square().mean(1) - 1).abs() <= 2e-2).all() and not x[:1000].any()
    api.dropout_fwd(x, 0.5, 7, out=x)
    first = (T - 3) * d  # a multiple of 8
    key = (7, 0)
    words = [philox_plain.philox(((first // 8 + i) & 0xffffffff, (first // 8 + i) >> 32, 0, 0), key) for i in range(64)]
    kept = np.array([[w & 0xffff, w >> 16] for four in words for w in four]).reshape(-1) >= 32768
    assert torch.equal((x[-3] != 0).cpu()[:512], torch.from_numpy(kept))


def test_graph_and_stream():
    x, res = (torch.randn(64, 512, device="cuda").to(BF) for _ in range(2))
    w = torch.randn(512, device="cuda").to(BF)
    seed = torch.tensor([5], device="cuda")
    out = [torch.zeros_like(x), None, torch.zeros_like(x), torch.zeros(64, device="cuda")]
    back = [torch.zeros_like(x), torch.zeros_like(x), torch.zeros(512, device="cuda")]
    ws = torch.empty(api.rmsnorm_workspace_bytes(64, 512), dtype=torch.uint8, device="cuda")

    def step():
        api.rmsnorm_fwd(x, w, residual=res, dropout=0.2, seed=seed, site=4, out=out)
        api.rmsnorm_bwd(out[0], out[2], w, out[3], dh=res, dropout=0.2, seed=seed, site=4, workspace=ws, out=back)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for s in (5, 6):
        seed.fill_(s)
        g.replay()
        torch.cuda.synchronize()
        fwd = api.rmsnorm_fwd(x, w, residual=res, dropout=0.2, seed=s, site=4)
        bwd = api.rmsnorm_bwd(fwd[0], fwd[2], w, fwd[3], dh=res, dropout=0.2, seed=s, site=4)
        for a, b in zip([*out, *back], [*fwd, *bwd]):
            assert a is None or torch.equal(a, b)


def test_rows_around_are_untouched():
    big = torch.full((8, 96), 3.0, device="cuda").to(BF)
    x = torch.randn(4, 64, device="cuda").to(BF)
    api.rmsnorm_fwd(x, out=(big[2:6, 16:80], None, None, torch.empty(4, device="cuda")))
    assert (big[:2] == 3).all() and (big[6:] == 3).all() and (big[:, :16] == 3).all() and (big[:, 80:] == 3).all()
    q8 = torch.full((8, 96), 1.0, device="cuda").to(torch.float8_e4m3fn)
    api.quantize_e4m3(x, out=(q8[2:6, 16:80], torch.empty(4, device="cuda")))
    f = q8.float()
    assert (f[:2] == 1).all() and (f[6:] == 1).all() and (f[:, :16] == 1).all() and (f[:, 80:] == 1).all()


def test_two_threads():
    """Calls of two widths from two host threads at once, each on its own stream: as one after the other."""
    import threading
    xs = [torch.randn(40, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d)) for d in (512, 4096)]
    want = [(api.rmsnorm_fwd(x)[0], api.rmsnorm_bwd(x, x, None, api.rmsnorm_fwd(x)[3])[0]) for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(x, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    y, _, _, rstd = api.rmsnorm_fwd(x)
                    dx, _, _ = api.rmsnorm_bwd(x, x, None, rstd)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(y, want[0]) and torch.equal(dx, want[1])):
                    wrong.append("another result")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=a) for a in zip(xs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
