"""Refusals and workspace sizes of the head cross entropy in pieces of the
vocabulary: everything here is decided on the host, before any launch."""
import ctypes

import pytest

from test_abi_host import _fake, lib  # noqa: F401  (fixture)

BF16, I32, I64 = 1, 2, 3


def _opts(ignore=-100, vocab=0, red=0, reserved=0, den=0.0):
    from backward_tcgen05_tma_gemms_gb300.api import TpsCeOptions
    return TpsCeOptions(ignore, vocab, red, reserved, den)


def _r(t):
    return bytes(t) if t is not None else None


def _fwd(lib, h=None, W=None, y=None, layout=0, o=None, loss=None, red=None, lse=None, ws=0x100000, n=1 << 40):
    return lib.tps_linear_ce_fwd(_r(h or _fake([8, 64], BF16)), _r(W or _fake([64, 512], BF16)),
                                 _r(y or _fake([8], I64)), layout, ctypes.byref(o) if o else None, _r(loss or _fake([8])), _r(red),
                                 _r(lse or _fake([8])), ctypes.c_void_p(ws), n, None)


def _bwd(lib, lse=None, g=None, o=None, dh=None, dW=None, ws=0x100000, n=1 << 40, none=False):
    return lib.tps_linear_ce_bwd(_r(_fake([8, 64], BF16)), _r(_fake([64, 512], BF16)), _r(_fake([8], I64)),
                                 _r(lse or _fake([8])), _r(g), 0, ctypes.byref(o) if o else None,
                                 None if none else _r(dh or _fake([8, 64])), None if none else _r(dW or _fake([64, 512])),
                                 ctypes.c_void_p(ws), n, None)


def test_forward_refusals(lib):  # noqa: F811
    assert _fwd(lib, W=_fake([65, 512], BF16)) == 1
    assert _fwd(lib, W=_fake([64, 0], BF16)) == 1
    assert _fwd(lib, W=_fake([64, 512])) == 3                     # fp32 head, bf16 hidden
    assert _fwd(lib, h=_fake([8, 64], I32), W=_fake([64, 512], I32)) == 3
    assert _fwd(lib, y=_fake([7], I64)) == 1
    assert _fwd(lib, y=_fake([8])) == 3
    assert _fwd(lib, y=_fake([8], I64, [2])) == 4
    assert _fwd(lib, loss=_fake([9])) == 1 and _fwd(lib, lse=_fake([8], BF16)) == 3
    assert _fwd(lib, layout=2) == 9
    assert _fwd(lib, o=_opts(vocab=513)) == 1 and _fwd(lib, o=_opts(red=3)) == 9
    assert _fwd(lib, o=_opts(den=-1.0)) == 9 and _fwd(lib, o=_opts(reserved=1)) == 9
    assert _fwd(lib, o=_opts(red=1), red=_fake([2])) == 1
    assert _fwd(lib, h=_fake([8, 64], BF16, [3, 2])) == 4         # no unit stride
    assert _fwd(lib, ws=0) == 6 and _fwd(lib, ws=0x100010) == 6 and _fwd(lib, n=64) == 6


def test_backward_refusals(lib):  # noqa: F811
    assert _bwd(lib, none=True) == 9
    assert _bwd(lib, lse=_fake([7])) == 1
    assert _bwd(lib, g=_fake([1])) == 1                           # one gradient for a loss for each token
    assert _bwd(lib, g=_fake([8]), o=_opts(red=2)) == 1           # and the other way round
    assert _bwd(lib, g=_fake([8], BF16)) == 3
    assert _bwd(lib, dh=_fake([8, 65])) == 1 and _bwd(lib, dh=_fake([8, 64], I32)) == 3
    assert _bwd(lib, dW=_fake([512, 64])) == 1
    assert _bwd(lib, n=1024) == 6 and _bwd(lib, ws=0x100001) == 6


def test_workspace_is_far_below_the_logits(lib):  # noqa: F811
    T, d, V = 8192, 4096, 128256
    f = lib.tps_linear_ce_workspace_bytes(T, d, V, BF16, 0, 0)
    b = lib.tps_linear_ce_workspace_bytes(T, d, V, BF16, 1, 0)
    assert f < T * V * 2 / 30 and b < T * V * 2 / 2.9
    assert lib.tps_linear_ce_workspace_bytes(T, d, V, BF16, 1, 256) < b
    least = lib.tps_linear_ce_workspace_bytes(8, 64, 512, BF16, 1, 1)
    assert _bwd(lib, n=least // 2) == 6
    for bad in ((-1, d, V, 1, 0, 0), (T, 0, V, 1, 0, 0), (T, d, 0, 1, 0, 0), (T, d, V, 2, 0, 0), (T, d, V, 1, 0, -1)):
        assert lib.tps_linear_ce_workspace_bytes(*bad) == 0


def test_python_refusals():
    import torch
    from backward_tcgen05_tma_gemms_gb300 import api
    h, W, y = torch.zeros(2, 8), torch.zeros(8, 16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="argument"):
        api.linear_ce_fwd(h, W, y, weight_layout="rows")
    with pytest.raises(ValueError, match="argument"):
        api.linear_ce_fwd(h, W, y, reduction="median")
    with pytest.raises(ValueError, match="GPU"):
        api.linear_ce_fwd(h, W, y)
