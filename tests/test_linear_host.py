"""Refusals of the linear product and its gradients: decided on the host, before any launch."""


import pytest

from test_abi_host import _fake, lib  # noqa: F401  (fixture)

F32, BF16, I32, I64, E4M3 = 0, 1, 2, 3, 4
OK, SHAPE, DTYPE, LAYOUT, WORKSPACE, ARG = 0, 1, 3, 4, 6, 9
IN_OUT, OUT_IN, NONE, SILU = 0, 1, -1, 3


def _r(t):
    return bytes(t) if t is not None else None


def fwd(lib, x=None, w=None, bias=None, res=None, act=NONE, layout=IN_OUT, xs=None, ws=None, z=None, y=None, room=None, n=0):
    return lib.tps_linear_fwd(_r(x or _fake([6, 64], BF16)), _r(w or _fake([64, 40], BF16)), _r(bias), _r(res), act, layout,
                              _r(xs), _r(ws), _r(z), _r(y or _fake([6, 40], BF16)), room, n, None)


def test_forward_refusals(lib):  # noqa: F811
    assert fwd(lib, layout=2) == ARG
    assert fwd(lib, act=4) == ARG
    assert fwd(lib, act=-2) == ARG
    assert fwd(lib, layout=OUT_IN) == SHAPE
    assert fwd(lib, x=_fake([6, 0], BF16), w=_fake([0, 40], BF16)) == SHAPE
    assert fwd(lib, w=_fake([64, 0], BF16), y=_fake([6, 0], BF16)) == SHAPE
    assert fwd(lib, x=_fake([64], BF16)) == SHAPE
    assert fwd(lib, x=_fake([6, 64])) == DTYPE                                   # of another type than W
    assert fwd(lib, x=_fake([6, 64], I32), w=_fake([64, 40], I32)) == DTYPE
    assert fwd(lib, x=_fake([6, 64], BF16, [128, 2])) == LAYOUT                  # no unit stride
    assert fwd(lib, bias=_fake([41])) == SHAPE
    assert fwd(lib, bias=_fake([40], I32)) == DTYPE
    assert fwd(lib, bias=_fake([40], BF16, [2])) == LAYOUT
    assert fwd(lib, res=_fake([6, 41], BF16)) == SHAPE
    assert fwd(lib, res=_fake([6, 40], E4M3)) == DTYPE
    assert fwd(lib, y=_fake([6, 41], BF16)) == SHAPE
    assert fwd(lib, y=_fake([6, 40], E4M3)) == DTYPE
    assert fwd(lib, y=_fake([6, 40], BF16, [1, 6])) == LAYOUT
    assert fwd(lib, y=_fake([6, 40], BF16, [20, 1])) == LAYOUT
    assert fwd(lib, z=_fake([5, 40], BF16)) == SHAPE
    assert fwd(lib, z=_fake([6, 40], BF16, [0, 1])) == LAYOUT
    assert fwd(lib, xs=_fake([6])) == ARG
    assert fwd(lib, x=_fake([1 << 31, 64], BF16)) == SHAPE
    assert fwd(lib, x=_fake([1 << 29, 64]), w=_fake([64, 40])) == SHAPE
    odd = _fake([6, 64], BF16)
    odd.data = 0x1001
    assert fwd(lib, x=odd) == LAYOUT
    assert fwd(lib, x=_fake([0, 64], BF16), y=_fake([0, 40], BF16)) == OK


def test_forward_refusals_e4m3(lib):  # noqa: F811
    x, w, xs, ws = _fake([6, 64], E4M3), _fake([40, 64], E4M3), _fake([6]), _fake([40])
    kw = dict(x=x, w=w, layout=OUT_IN)
    assert fwd(lib, **kw) == ARG
    assert fwd(lib, **kw, xs=xs) == ARG
    assert fwd(lib, **kw, xs=ws, ws=ws) == SHAPE
    assert fwd(lib, **kw, xs=xs, ws=xs) == SHAPE
    assert fwd(lib, **kw, xs=_fake([6], BF16), ws=ws) == DTYPE
    assert fwd(lib, x=x, w=_fake([64, 40], E4M3), xs=xs, ws=ws) == LAYOUT        # (in, out)
    assert fwd(lib, x=_fake([6, 50], E4M3), w=_fake([40, 50], E4M3), layout=OUT_IN, xs=xs, ws=ws) == LAYOUT
    off = _fake([6, 64], E4M3)
    off.data = 0x1008
    assert fwd(lib, x=off, w=w, layout=OUT_IN, xs=xs, ws=ws) == LAYOUT


def test_workspace(lib):  # noqa: F811
    """bf16 that starts off 16 bytes, and fp32, are laid out in a workspace."""
    assert lib.tps_linear_workspace_bytes(6, 64, 40, BF16, 0) == 0
    assert lib.tps_linear_workspace_bytes(6, 64, 40, E4M3, 0) == 0
    assert lib.tps_linear_workspace_bytes(-1, 64, 40, BF16, 1) == 0
    assert lib.tps_linear_workspace_bytes(6, 0, 40, F32, 1) == 0
    off = _fake([6, 64], BF16)
    off.data = 0x1002
    assert fwd(lib, x=off) == WORKSPACE
    f32 = dict(x=_fake([600, 64]), w=_fake([64, 40]), y=_fake([600, 40]))
    need = lib.tps_linear_workspace_bytes(600, 64, 40, F32, 0)
    assert need >= (600 + 40) * 64 * 6
    assert fwd(lib, **f32) == WORKSPACE
    assert fwd(lib, **f32, room=0x1000, n=need - 256) == WORKSPACE
    assert fwd(lib, **f32, room=0x1080, n=need) == WORKSPACE


def test_backward_refusals(lib):  # noqa: F811
    def bwd(x=None, w=None, dy=None, z=None, act=NONE, layout=IN_OUT, dx=None, dw=None, db=None, room=None, n=0):
        return lib.tps_linear_bwd(_r(x or _fake([6, 64], BF16)), _r(w or _fake([64, 40], BF16)),
                                  _r(dy or _fake([6, 40], BF16)), _r(z), act, layout, _r(dx), _r(dw), _r(db), room, n, None)
    assert bwd(x=_fake([6, 64], E4M3), w=_fake([64, 40], E4M3)) == DTYPE
    assert bwd(dy=_fake([6, 41], BF16)) == SHAPE
    assert bwd(dy=_fake([6, 40], E4M3)) == DTYPE
    assert bwd(act=SILU) == ARG
    assert bwd(z=_fake([6, 40], BF16)) == ARG
    assert bwd(act=SILU, z=_fake([6, 41], BF16)) == SHAPE
    assert bwd(act=7, z=_fake([6, 40], BF16)) == ARG
    assert bwd(dx=_fake([6, 40], BF16)) == SHAPE
    assert bwd(dx=_fake([6, 64], E4M3)) == DTYPE
    assert bwd(dx=_fake([6, 64], BF16, [0, 1])) == LAYOUT
    assert bwd(dw=_fake([40, 64], BF16)) == SHAPE
    assert bwd(dw=_fake([64, 40], I64)) == DTYPE
    assert bwd(dw=_fake([64, 40], BF16, [0, 1])) == LAYOUT
    assert bwd(db=_fake([41])) == SHAPE
    assert bwd(db=_fake([40], I32)) == DTYPE
    assert bwd(db=_fake([40])) == WORKSPACE
    assert bwd(act=SILU, z=_fake([6, 40], BF16), dx=_fake([6, 64], BF16)) == WORKSPACE


def test_binding_refusals(lib):  # noqa: F811
    import torch
    from backward_tcgen05_tma_gemms_gb300 import api
    x, W = torch.zeros(4, 8), torch.zeros(8, 8)
    for call in (lambda: api.linear_fwd(x, W), lambda: api.linear_bwd(x, W, x)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
    with pytest.raises(ValueError, match="argument"):
        api.linear_fwd(x, W, act="relu")
    with pytest.raises(ValueError, match="shape"):
        api.linear_fwd(x, W[0])


def test_vectors_off_their_elements(lib):  # noqa: F811
    """A vector that does not start at a multiple of its element's size is refused."""
    def off(n, dtype=F32, by=2):
        t = _fake([n], dtype)
        t.data += by
        return t
    assert fwd(lib, bias=off(40)) == LAYOUT and fwd(lib, bias=off(40, BF16, 1)) == LAYOUT
    codes = dict(x=_fake([6, 64], E4M3), w=_fake([40, 64], E4M3), layout=OUT_IN)
    assert fwd(lib, **codes, xs=off(6), ws=_fake([40])) == LAYOUT
    assert fwd(lib, **codes, xs=_fake([6]), ws=off(40)) == LAYOUT
    for db in (off(40), off(40, BF16, 1)):
        assert lib.tps_linear_bwd(_r(_fake([6, 64], BF16)), _r(_fake([64, 40], BF16)), _r(_fake([6, 40], BF16)), None, NONE,
                                  IN_OUT, None, None, _r(db), 0x1000, 1 << 20, None) == LAYOUT


def test_weight_gradient_that_overlaps(lib):  # noqa: F811
    """Every element of dW has a place of its own, also where W is a vector."""
    def bwd(w, dw):
        K, N = w
        return lib.tps_linear_bwd(_r(_fake([6, K], BF16)), _r(_fake(list(w), BF16)), _r(_fake([6, N], BF16)), None, NONE,
                                  IN_OUT, None, _r(_fake(list(w), F32, dw)), None, None, 0, None)
    for w, dw in (((64, 40), [0, 1]), ((64, 40), [39, 1]), ((64, 40), [1, 63]), ((64, 1), [0, 1]), ((64, 1), [-1, 1]),
                  ((1, 40), [40, 0]), ((1, 40), [40, -1])):
        assert bwd(w, dw) == LAYOUT, (w, dw)
    # fine: refused at last for want of a workspace for x and W, which start off 16 bytes
    for w, dw in (((64, 1), [1, 1]), ((64, 1), [5, 1]), ((1, 40), [40, 1]), ((1, 40), [0, 1]), ((64, 1), [1, 0])):
        K, N = w
        x, W = _fake([6, K], BF16), _fake(list(w), BF16)
        x.data = W.data = 0x1002
        assert lib.tps_linear_bwd(_r(x), _r(W), _r(_fake([6, N], BF16)), None, NONE, IN_OUT, None, _r(_fake(list(w), F32, dw)),
                                  None, None, 0, None) == WORKSPACE, (w, dw)


def test_long_fp32_contractions(lib):  # noqa: F811
    """Six products over K must count below 2^31: what does not is refused before a workspace is asked for."""
    most = ((1 << 31) - 1) // 6
    for K, want in ((most + 1, SHAPE), (most, WORKSPACE)):
        assert fwd(lib, x=_fake([9, K]), w=_fake([K, 1]), y=_fake([9, 1])) == want

    def bwd(T, K, N, dx, dw):
        return lib.tps_linear_bwd(_r(_fake([T, K])), _r(_fake([K, N])), _r(_fake([T, N])), None, NONE, IN_OUT,
                                  _r(_fake([T, K])) if dx else None, _r(_fake([K, N])) if dw else None, None, None, 0, None)
    for n, want in ((most + 1, SHAPE), (most, WORKSPACE)):
        assert bwd(2, 1, n, True, False) == want and bwd(n, 1, 2, False, True) == want
        assert bwd(2, n, 1, True, True) == WORKSPACE  # K is no contraction backwards
    assert bwd(most + 1, 1, 2, True, False) == WORKSPACE
    # bf16 runs one product
    x, w = _fake([9, most + 1], BF16, [1 << 29, 1]), _fake([most + 1, 1], BF16)
    x.data = 0x1002
    assert fwd(lib, x=x, w=w, y=_fake([9, 1], BF16)) == WORKSPACE
