"""The generator behind the dropout mask against its published vectors, and
refusals of the norm, dropout and e4m3 rows: decided on the host, before any launch."""
import math
import struct

import pytest
import torch

import philox_plain
from test_abi_host import _fake, lib  # noqa: F401  (fixture)

F32, BF16, I32, I64, E4M3 = 0, 1, 2, 3, 4
OK, SHAPE, DTYPE, LAYOUT, WORKSPACE, ARG = 0, 1, 3, 4, 6, 9


def _r(t):
    return bytes(t) if t is not None else None


def _drop(p, seed=1, ptr=0, site=0):
    return struct.pack("=dQQQ", p, seed, ptr, site)


def test_plain_generator_gives_the_published_vectors():
    """The known answers that the generator's authors publish for it."""
    full = [0xffffffff] * 6
    pi = [0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344, 0xa4093822, 0x299f31d0]
    for words, want in (([0] * 6, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
                        (full, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
                        (pi, [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])):
        assert philox_plain.philox(words[:4], words[4:]) == want


def test_plain_mask_keeps_its_share():
    """16384 draws of probability 0.25: within five deviations of the share."""
    n, p = 16384, 0.25
    kept = (philox_plain.mask((n,), p, 77, 3) > 0).mean()
    assert abs(kept - (1 - p)) <= 5 * math.sqrt(p * (1 - p) / n)
    assert (philox_plain.draws(64, 1, 0) != philox_plain.draws(64, 1, 1)).any()
    assert (philox_plain.draws(64, 1, 0) != philox_plain.draws(64, 2, 0)).any()


def fwd(lib, x=None, res=None, w=None, eps=1e-6, drop=None, h=None, y=None, scale=None, rstd=None):
    x = x or _fake([6, 64], BF16)
    return lib.tps_rmsnorm_fwd(_r(x), _r(res), _r(w), eps, drop, _r(h), _r(y or _fake([6, 64], BF16)), _r(scale),
                               _r(rstd or _fake([6])), None)


def test_norm_refusals(lib):  # noqa: F811
    assert fwd(lib, x=_fake([64], BF16)) == SHAPE                                  # not rows
    assert fwd(lib, x=_fake([6, 64], I32)) == DTYPE
    assert fwd(lib, x=_fake([6, 64], E4M3)) == DTYPE
    assert fwd(lib, x=_fake([6, 64], BF16, [1, 6])) == LAYOUT                      # columns are contiguous
    assert fwd(lib, x=_fake([2, 3, 64], BF16, [999, 64, 1])) == LAYOUT             # rows without one pitch
    assert fwd(lib, y=_fake([6, 63], BF16)) == SHAPE
    assert fwd(lib, y=_fake([6, 64], BF16, [32, 1])) == LAYOUT                     # rows overlap
    assert fwd(lib, y=_fake([6, 64], BF16, [0, 1])) == LAYOUT
    assert fwd(lib, y=_fake([6, 64], E4M3)) == ARG                                 # without its scale
    assert fwd(lib, scale=_fake([6])) == ARG                                       # without codes
    assert fwd(lib, y=_fake([6, 64], E4M3), scale=_fake([5])) == SHAPE
    assert fwd(lib, y=_fake([6, 64], E4M3), scale=_fake([6], BF16)) == DTYPE
    assert fwd(lib, w=_fake([63], BF16)) == SHAPE
    assert fwd(lib, w=_fake([64], E4M3)) == DTYPE
    assert fwd(lib, w=_fake([64], BF16, [2])) == LAYOUT
    assert fwd(lib, rstd=_fake([5])) == SHAPE
    assert fwd(lib, rstd=_fake([6], BF16)) == DTYPE
    for eps in (-1e-6, math.nan, math.inf):
        assert fwd(lib, eps=eps) == ARG
    assert fwd(lib, res=_fake([6, 64], BF16)) == ARG                               # the sum is wanted
    assert fwd(lib, res=_fake([6, 64], BF16), h=_fake([6, 64])) == DTYPE           # of the residual's type
    assert fwd(lib, res=_fake([5, 64], BF16), h=_fake([6, 64], BF16)) == SHAPE
    assert fwd(lib, h=_fake([6, 64], BF16)) == ARG                                 # it is the input
    assert fwd(lib, drop=_drop(0.1)) == ARG
    for p in (-0.1, 1.1, math.nan):
        assert fwd(lib, drop=_drop(p), h=_fake([6, 64], BF16)) == ARG
    assert fwd(lib, drop=_drop(0.1, ptr=0x1001), h=_fake([6, 64], BF16)) == LAYOUT
    odd = _fake([6, 64], BF16)
    odd.data = 0x1001
    assert fwd(lib, x=odd) == LAYOUT
    assert fwd(lib, x=_fake([1 << 31, 1], BF16)) == SHAPE
    assert fwd(lib, x=_fake([6, 0], BF16), y=_fake([6, 0], BF16)) == SHAPE         # no mean of nothing
    assert fwd(lib, x=_fake([0, 64], BF16), y=_fake([0, 64], BF16), rstd=_fake([0])) == OK


def test_norm_backward_refusals(lib):  # noqa: F811
    def bwd(dy=None, h=None, w=None, rstd=None, dh=None, drop=None, dsum=None, dx=None, dw=None, ws=0x1000, n=1 << 20):
        return lib.tps_rmsnorm_bwd(_r(dy or _fake([6, 64], BF16)), _r(h or _fake([6, 64], BF16)), _r(w),
                                   _r(rstd or _fake([6])), _r(dh), drop, _r(dsum), _r(dx), _r(dw), ws, n, None)
    assert bwd(dy=_fake([6, 64], E4M3)) == DTYPE
    assert bwd(h=_fake([6, 65], BF16)) == SHAPE
    assert bwd(rstd=_fake([7])) == SHAPE
    assert bwd(w=_fake([65])) == SHAPE
    assert bwd(dh=_fake([6, 64])) == DTYPE
    assert bwd(dsum=_fake([6, 64])) == DTYPE
    assert bwd(dsum=_fake([6, 64], BF16, [0, 1])) == LAYOUT
    assert bwd(dx=_fake([7, 64], BF16)) == SHAPE
    assert bwd(dx=_fake([6, 64], E4M3)) == DTYPE
    assert bwd(dw=_fake([64], BF16)) == DTYPE
    assert bwd(dw=_fake([63])) == SHAPE
    assert bwd(drop=_drop(2.0)) == ARG
    need = lib.tps_rmsnorm_workspace_bytes(6, 64)
    assert need >= 6 * 64 * 4
    assert bwd(dw=_fake([64]), n=need - 1) == WORKSPACE
    assert bwd(dw=_fake([64]), ws=0x1010) == WORKSPACE
    assert bwd(dw=_fake([64]), ws=None) == WORKSPACE
    assert lib.tps_rmsnorm_workspace_bytes(-1, 64) == 0
    # rows 1 << 20: no more partial sums than blocks
    assert lib.tps_rmsnorm_workspace_bytes(1 << 20, 64) < (1 << 20) * 64


def test_dropout_and_quantize_refusals(lib):  # noqa: F811
    def drop(x=None, res=None, o=_drop(0.1), y=None):
        return lib.tps_dropout_fwd(_r(x or _fake([6, 64], BF16)), _r(res), o, _r(y or _fake([6, 64], BF16)), None)
    assert drop(o=None) == ARG
    assert drop(o=_drop(1.5)) == ARG
    assert drop(x=_fake([6, 64], I64)) == DTYPE
    assert drop(res=_fake([6, 63], BF16)) == SHAPE
    assert drop(y=_fake([6, 64], E4M3)) == DTYPE
    assert drop(y=_fake([6, 64], BF16, [8, 1])) == LAYOUT
    assert drop(x=_fake([0, 64], BF16), y=_fake([0, 64], BF16)) == OK
    assert lib.tps_dropout_bwd(_r(_fake([6, 64])), _drop(-1.0), _r(_fake([6, 64])), None) == ARG

    def quant(x=None, q=None, scale=None):
        return lib.tps_quantize_e4m3(_r(x or _fake([6, 64], BF16)), _r(q or _fake([6, 64], E4M3)),
                                     _r(scale or _fake([6])), None)
    assert quant(q=_fake([6, 64], BF16)) == DTYPE
    assert quant(x=_fake([6, 64], E4M3)) == DTYPE
    assert quant(q=_fake([6, 32], E4M3)) == SHAPE
    assert quant(scale=_fake([7])) == SHAPE
    assert quant(x=_fake([0, 64]), q=_fake([0, 64], E4M3), scale=_fake([0])) == OK


def test_binding_refusals(lib):  # noqa: F811
    from backward_tcgen05_tma_gemms_gb300 import api
    x = torch.zeros(4, 8)
    for call in (lambda: api.rmsnorm_fwd(x), lambda: api.dropout_fwd(x, 0.5, 1), lambda: api.quantize_e4m3(x),
                 lambda: api.rmsnorm_bwd(x, x, None, torch.zeros(4))):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
    for seed in (torch.zeros(2, dtype=torch.int64), torch.zeros(1)):
        with pytest.raises(ValueError, match="seed"):
            api.dropout_fwd(x, 0.5, seed)
    for call in (lambda: api.rmsnorm_fwd(None), lambda: api.rmsnorm_fwd(x, weight=3), lambda: api.dropout_fwd(x, 0.5, "1"),
                 lambda: api.quantize_e4m3([1.0]), lambda: api.rmsnorm_fwd(x, out_dtype="f32")):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_vectors_off_their_elements(lib):  # noqa: F811
    """A vector that does not start at a multiple of its element's size is refused."""
    def off(n, dtype=F32, by=2):
        t = _fake([n], dtype)
        t.data += by
        return t
    x = _fake([6, 64], BF16)
    assert fwd(lib, rstd=off(6)) == LAYOUT
    assert fwd(lib, w=off(64)) == LAYOUT and fwd(lib, w=off(64, BF16, 1)) == LAYOUT
    assert fwd(lib, y=_fake([6, 64], E4M3), scale=off(6)) == LAYOUT
    assert lib.tps_quantize_e4m3(_r(x), _r(_fake([6, 64], E4M3)), _r(off(6)), None) == LAYOUT
    for rstd, dw in ((off(6), None), (_fake([6]), off(64))):
        assert lib.tps_rmsnorm_bwd(_r(x), _r(x), None, _r(rstd), None, None, None, None, _r(dw), 0x1000, 1 << 20, None) == LAYOUT


def test_quantize_rows_without_elements(lib):  # noqa: F811
    """Rows of nothing have no largest magnitude."""
    def quant(T, d, dtype=BF16):
        return lib.tps_quantize_e4m3(_r(_fake([T, d], dtype)), _r(_fake([T, d], E4M3)), _r(_fake([T])), None)
    for dtype in (BF16, F32):
        assert quant(6, 0, dtype) == SHAPE and quant(1, 0, dtype) == SHAPE
        assert quant(0, 0, dtype) == OK


def test_leading_extents_of_one(lib):  # noqa: F811
    """Rows with one pitch are rows with one pitch whatever the strides of extents of one are: the last tokens of
    a batch, [:, -1:].  What passes the views is refused for its eps, before any launch."""
    def view(shape, strides):
        return fwd(lib, x=_fake(shape, BF16, strides), eps=-1.0)
    assert view([6, 1, 64], [128, 64, 1]) == ARG
    assert view([1, 6, 64], [999, 128, 1]) == ARG
    assert view([6, 1, 64], [128, 999, 1]) == ARG
    assert view([2, 1, 3, 64], [384, 7, 128, 1]) == ARG
    assert view([2, 3, 1, 64], [384, 128, 7, 1]) == ARG
    assert view([3, 0, 64], [64, 64, 1]) == ARG
    assert view([2, 3, 64], [0, 0, 1]) == ARG
    assert view([2, 3, 64], [192, 0, 1]) == LAYOUT
    assert view([2, 3, 64], [0, 64, 1]) == LAYOUT
    assert view([2, 1, 3, 64], [999, 192, 64, 1]) == LAYOUT
    assert view([2, 3, 1, 64], [999, 64, 64, 1]) == LAYOUT


def test_one_tensor_for_both_gradients(lib):  # noqa: F811
    """dSum and dX differ by the dropout: they cannot be one tensor then.  What passes is refused for its
    workspace, before any launch."""
    def bwd(drop, dsum, dx, h=BF16):
        return lib.tps_rmsnorm_bwd(_r(_fake([6, 64], BF16)), _r(_fake([6, 64], h)), None, _r(_fake([6])), None, drop, _r(dsum),
                                   _r(dx), _r(_fake([64])), None, 0, None)
    t, other = _fake([6, 64], BF16), _fake([6, 64], BF16)
    other.data = 0x9000
    assert bwd(_drop(0.25), t, t) == ARG
    assert bwd(_drop(0.25), t, other) == WORKSPACE
    assert bwd(None, t, t) == WORKSPACE and bwd(_drop(0.0), t, t) == WORKSPACE
    assert bwd(None, _fake([6, 64]), t, h=F32) == ARG                               # fp32 and bf16 in one place
    assert bwd(None, t, _fake([6, 64], BF16, [128, 1])) == ARG
    assert bwd(_drop(0.25), t, None) == WORKSPACE and bwd(_drop(0.25), None, t) == WORKSPACE
