"""Rotary positions (rope_fwd / rope_bwd) against the rotation in float64.

Bounds: the angle is off by pi 2^-25 (its fraction of a turn as a float) and
sincospif by two units, 2^-21 together; a turned element adds two products,
so it is off by (|a| + |b|) amp (2^-21 + 2^-22), and by half a step of its
type (2^-8 for bf16, 2^-24 for fp32)."""
import math

import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, context=4096.0):
    if scaling == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    amp = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        amp = 0.1 * math.log(factor) + 1
        lo = max(math.floor(rot * math.log(context / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
        hi = min(math.ceil(rot * math.log(context / (2 * math.pi)) / (2 * math.log(base))), rot - 1)
        for i, x in enumerate(f):
            r = min(1, max(0, (i - lo) / max(hi - lo, 1e-3)))
            f[i] = x / factor * r + x * (1 - r)
    return f, amp


def reference(x, pos, f, amp, rot, inter, sign):
    """x (rows, H, D) and its bound."""
    a = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = amp * a.cos()[:, None], sign * amp * a.sin()[:, None]
    d = x.double()
    i = torch.arange(rot // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    out, err = d.clone(), torch.zeros_like(d)
    out[..., lo] = d[..., lo] * c - d[..., hi] * s
    out[..., hi] = d[..., hi] * c + d[..., lo] * s
    err[..., lo] = err[..., hi] = (d[..., lo].abs() + d[..., hi].abs()) * amp * (2.0 ** -21 + 2.0 ** -22)
    turned = torch.zeros(x.shape[-1], device=x.device, dtype=torch.bool)
    turned[:rot] = True
    return out, err + HALF[x.dtype] * (out.abs() + err) * turned


def check(B, S, H, Hk, D, rot, dtype, inter=False, scaling="none", factor=1.0, far=0, pos_dtype=torch.int64, four=True,
          in_place=False, packed=False, shared=False, pos=None):
    g = torch.Generator().manual_seed(B + S + H + D)
    if packed:
        x = torch.randn(B, S, H + 2 * Hk, D, generator=g).to(dtype).cuda()
        q, k = x[:, :, :H], x[:, :, H:H + Hk]
    else:
        q, k = (torch.randn(B, S, n, D, generator=g).to(dtype).cuda() for n in (H, Hk))
    if pos is None:
        pos = far + torch.arange(S).expand(1 if shared else B, S) + (0 if shared else torch.arange(B)[:, None])
    pos = pos.to(pos_dtype).cuda().contiguous()
    plan = api.rope_plan(rot, interleaved=inter, scaling=scaling, factor=factor, original_context=4096)
    f, amp = frequencies(rot, scaling=scaling, factor=factor)
    rows = pos.expand(B, S).reshape(-1)
    for turn, sign in ((api.rope_fwd, 1), (api.rope_bwd, -1)):
        a, b = (q.clone(), k.clone()) if in_place else (q, k)
        if not four:
            a, b, p = a.flatten(0, 1), b.flatten(0, 1), rows
        else:
            p = pos[0].contiguous() if shared else pos
        out = turn(plan, a, b, p, out=(a, b) if in_place else None)
        for got, x in zip(out, (q, k)):
            want, bound = reference(x.reshape(B * S, -1, D), rows, f, amp, rot, inter, sign)
            diff = (got.reshape(B * S, -1, D).double() - want).abs()
            assert (diff <= bound).all(), f"{turn.__name__}: {(diff - bound).max().item():.3e} over"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,S,H,Hk,D,rot", [(1, 1, 1, 1, 2, 2), (1, 3, 5, 1, 6, 4), (2, 7, 8, 2, 64, 64), (1, 129, 3, 3, 80, 80),
                                            (3, 33, 4, 2, 96, 64), (1, 40, 9, 1, 128, 32), (2, 5, 2, 1, 256, 256),
                                            (1, 17, 4, 4, 512, 512), (1, 11, 2, 2, 88, 64), (1, 9, 3, 1, 72, 16), (70, 1, 32, 8, 128, 128)])
def test_sizes(B, S, H, Hk, D, rot, dtype, inter):
    check(B, S, H, Hk, D, rot, dtype, inter)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("far", [0, 1 << 17, 1 << 20, (1 << 31) - 40])
def test_far_positions_and_scalings(scaling, far):
    # at 2^31 the reference's own double angle is off by 2^31 2^-53 2 pi < 2^-19.3 radians of 1
    if far > 1 << 30:
        plan = api.rope_plan(2, base=3.0)
        x = torch.randn(30, 2, 2, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        pos = torch.arange(30, device="cuda") + far
        y, _ = api.rope_fwd(plan, x, None, pos)
        want, bound = reference(x, pos, [1.0], 1.0, 2, False, 1)
        assert ((y.double() - want).abs() <= bound + x.double().abs().sum(-1, keepdim=True) * 2.0 ** -19).all()
        return
    check(2, 31, 4, 2, 128, 128, torch.bfloat16, scaling=scaling, factor=8.0, far=far)
    check(2, 31, 4, 2, 64, 64, torch.float32, True, scaling=scaling, factor=8.0, far=far)


@pytest.mark.parametrize("kw", [dict(in_place=True), dict(packed=True), dict(four=False), dict(pos_dtype=torch.int32),
                                dict(shared=True), dict(in_place=True, four=False, inter=True)], ids=str)
@pytest.mark.parametrize("rot", [128, 64])
def test_layouts(kw, rot):
    check(3, 21, 6, 3, 128, rot, torch.bfloat16, **kw)


def test_negative_positions_and_zero():
    check(1, 4, 2, 1, 64, 64, torch.float32, pos=torch.tensor([[-5, -1, 0, 3]]))


def test_unaligned_views():
    """Heads that start off 16 bytes, and a misaligned row pitch, go one pair at a time."""
    x = torch.randn(20, 3 * 66 + 1, device="cuda").to(torch.bfloat16)
    q = x[:, 1:].unflatten(1, (3, 66))
    plan = api.rope_plan(64)
    pos = torch.arange(20, device="cuda")
    y, _ = api.rope_fwd(plan, q, None, pos)
    want, bound = reference(q, pos, *frequencies(64), 64, False, 1)
    assert ((y.double() - want).abs() <= bound).all()


def test_two_dimensional_heads_and_round_trip():
    q = torch.randn(50, 8 * 64, device="cuda")
    plan, pos = api.rope_plan(64), torch.arange(50, device="cuda")
    y, none = api.rope_fwd(plan, q, None, pos, head_dim=64)
    z, _ = api.rope_bwd(plan, y, None, pos, head_dim=64)
    assert none is None and y.shape == q.shape
    assert (z - q).abs().max() <= 8 * 2.0 ** -20 * q.abs().max()  # the rotation and its transpose


def test_backward_is_the_transposed_forward():
    """<rope(x), y> = <x, rope_bwd(y)>, amplitude included."""
    plan, pos = api.rope_plan(64, scaling="yarn", factor=16.0, original_context=4096), torch.arange(30, device="cuda") * 999
    x, y = torch.randn(30, 2, 96, device="cuda"), torch.randn(30, 2, 96, device="cuda")
    a = (api.rope_fwd(plan, x, None, pos)[0].double() * y.double()).sum()
    b = (x.double() * api.rope_bwd(plan, y, None, pos)[0].double()).sum()
    assert abs(a - b) <= 2.0 ** -19 * 2 * (x.double().abs() * y.double().abs()).sum() + 1e-3


def test_empty_and_neighbours_untouched():
    plan = api.rope_plan(32)
    q = torch.empty(0, 4, 32, device="cuda")
    assert api.rope_fwd(plan, q, None, torch.empty(0, dtype=torch.int64, device="cuda"))[0].shape == (0, 4, 32)
    big = torch.full((5, 4, 48), 3.0, device="cuda")
    x = torch.randn(5, 2, 32, device="cuda")
    api.rope_fwd(plan, x, None, torch.arange(5, device="cuda"), out=(big[:, 1:3, 8:40], None))
    assert (big[:, 0] == 3).all() and (big[:, 3] == 3).all() and (big[..., :8] == 3).all() and (big[..., 40:] == 3).all()


def test_past_32_bit_offsets():
    """4.3 GB of heads: the last tokens turn like any others."""
    T, H, D = 131072 + 3, 64, 256
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    q[-5:] = torch.randn(5, H, D, device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, device="cuda")
    plan = api.rope_plan(D)
    want, bound = reference(q[-5:], pos[-5:], *frequencies(D), D, False, 1)
    y, _ = api.rope_fwd(plan, q, None, pos, out=(q, None))
    assert ((y[-5:].double() - want).abs() <= bound).all() and not y[:1000].any()


def test_graph_and_stream():
    plan = api.rope_plan(128)
    q, k = torch.randn(64, 8, 128, device="cuda"), torch.randn(64, 2, 128, device="cuda")
    pos = torch.arange(64, device="cuda")
    want = api.rope_fwd(plan, q, k, pos)
    out = (torch.zeros_like(q), torch.zeros_like(k))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.rope_fwd(plan, q, k, pos, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
