"""Refusals of the rotary positions and of the optimizer step, and the rotary
plan itself: decided on the host, before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_abi_host import _fake, lib  # noqa: F401  (fixture)

BF16, I32, I64, E4M3 = 1, 2, 3, 4


def _r(t):
    return bytes(t) if t is not None else None


def test_rope_plan_frequencies(lib):  # noqa: F811
    from backward_tcgen05_tma_gemms_gb300 import api
    for rot, base in ((2, 10.0), (64, 10000.0), (128, 500000.0), (512, 10000.0)):
        plan = api.rope_plan(rot, base=base)
        for i in range(rot // 2):
            want = base ** (-2 * i / rot) / (2 * math.pi)
            # cut to a multiple of 2^-64; the double before it is good to a few units of 2^-53
            assert abs(plan.turns[i] / 2.0 ** 64 - want) <= 2.0 ** -64 + want * 2.0 ** -48
        assert plan.amplitude == 1.0
    a, b = api.rope_plan(64), api.rope_plan(64, scaling="linear", factor=4.0)
    assert all(abs(a.turns[i] / 4 - b.turns[i]) <= 1 + a.turns[i] * 2.0 ** -50 for i in range(32))
    y = api.rope_plan(64, scaling="yarn", factor=4.0, original_context=2048)
    assert y.turns[0] == a.turns[0] and abs(y.turns[31] - a.turns[31] / 4) <= 1 + a.turns[31] * 2.0 ** -50
    assert abs(y.amplitude - (0.1 * math.log(4.0) + 1)) < 1e-6
    assert api.rope_plan(64, scaling="yarn", factor=4.0, original_context=2048, attention_factor=1.5).amplitude == 1.5


def test_rope_plan_refusals(lib):  # noqa: F811
    from backward_tcgen05_tma_gemms_gb300 import api
    for rot in (0, -2, 3, 514):
        with pytest.raises(ValueError, match="shape"):
            api.rope_plan(rot)
    with pytest.raises(ValueError, match="argument"):
        api.rope_plan(64, scaling="cubic")
    for kw in (dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(scaling="linear", factor=0.5),
               dict(scaling="ntk", factor=math.inf), dict(scaling="yarn", factor=2.0),
               dict(scaling="yarn", factor=2.0, original_context=4096, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(api.TpsError) as e:
            api.rope_plan(64, **kw)
        assert e.value.code == 9
    with pytest.raises(ValueError, match="shape"):
        api.rope_plan(2, scaling="ntk", factor=2.0)


def test_rope_refusals(lib):  # noqa: F811
    from backward_tcgen05_tma_gemms_gb300 import api
    plan = api.rope_plan(64)

    def call(q=None, k=None, pos=None, qo=None, ko=None, plan=plan, no_k=False):
        q, qo = q or _fake([6, 4, 64], BF16), qo or _fake([6, 4, 64], BF16)
        k, ko = (None, None) if no_k else (k or _fake([6, 2, 64], BF16), ko or _fake([6, 2, 64], BF16))
        return lib.tps_rope_fwd(ctypes.byref(plan), _r(q), _r(k), _r(pos or _fake([6], I64)), _r(qo), _r(ko), None)
    assert call(q=_fake([6, 256], BF16)) == 1                              # 2-D
    assert call(q=_fake([6, 4, 32], BF16), qo=_fake([6, 4, 32], BF16), no_k=True) == 1   # heads narrower than the plan
    assert call(qo=_fake([6, 4, 65], BF16)) == 1 and call(qo=_fake([6, 4, 64])) == 3
    assert call(k=_fake([5, 2, 64], BF16)) == 1 and call(k=_fake([6, 2, 64])) == 3
    assert call(ko=_fake([6, 3, 64], BF16)) == 1 and call(ko=_fake([6, 2, 64])) == 3
    assert call(q=_fake([6, 4, 64], BF16, [256, 1, 4])) == 4               # head not contiguous
    assert call(q=_fake([6, 4, 64], I32)) == 3
    assert call(pos=_fake([5], I64)) == 1 and call(pos=_fake([6])) == 3 and call(pos=_fake([6], I64, [2])) == 4
    assert lib.tps_rope_fwd(ctypes.byref(plan), _r(_fake([6, 4, 64])), _r(_fake([6, 2, 64])), _r(_fake([6], I64)),
                            _r(_fake([6, 4, 64])), None, None) == 9        # K without K out
    assert lib.tps_rope_fwd(None, _r(_fake([6, 4, 64])), None, _r(_fake([6], I64)), _r(_fake([6, 4, 64])), None, None) == 9
    assert call(plan=api.RopePlan()) == 9                                  # never initialised


def _row(**kw):
    from backward_tcgen05_tma_gemms_gb300.api import _ADAMW_ROW
    t = np.zeros(1, _ADAMW_ROW)
    for k, v in dict(dict(param=0x1000, grad=0x2000, m=0x3000, v=0x4000, numel=10), **kw).items():
        t[k] = v
    return t


def _step(lib, row, **kw):
    from backward_tcgen05_tma_gemms_gb300.api import TpsAdamwHyper
    h = dict(dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, seed=0, stochastic=0), **kw)
    scale = h.pop("scale", None)
    return lib.tps_adamw_step(row.ctypes.data, len(row), ctypes.byref(TpsAdamwHyper(**h)), scale, None, None)


def test_adamw_refusals(lib):  # noqa: F811
    for bad in (dict(lr=-1.0), dict(lr=math.nan), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1e-9), dict(eps=math.inf),
                dict(step=0), dict(weight_decay=math.inf), dict(beta2=math.nan)):
        assert _step(lib, _row(), **bad) == 9, bad
    assert _step(lib, _row(numel=-1)) == 1 and _step(lib, _row(place=128)) == 9 and _step(lib, _row(place=-256)) == 9
    assert _step(lib, _row(param_dtype=I32)) == 3 and _step(lib, _row(grad_dtype=E4M3)) == 3
    assert _step(lib, _row(state_dtype=BF16)) == 3
    assert _step(lib, _row(master=0x5000)) == 3                            # master of fp32 weights
    assert _step(lib, _row(param=0)) == 9 and _step(lib, _row(v=0)) == 9
    assert _step(lib, _row(state_dtype=E4M3)) == 9                         # scales missing
    assert _step(lib, _row(m_scale=0x6000, v_scale=0x7000)) == 9           # scales of fp32 moments
    assert _step(lib, _row(param=0x1002)) == 4 and _step(lib, _row(grad=0x2001, grad_dtype=BF16)) == 4
    assert _step(lib, _row(), scale=0x1001) == 4
    assert lib.tps_adamw_step(None, 1, None, None, None, None) == 9
    assert _step(lib, _row(numel=0, param=0)) == 0                         # nothing to do: nothing launched


def test_grad_norm_refusals(lib):  # noqa: F811
    from backward_tcgen05_tma_gemms_gb300.api import _SPAN_ROW

    def call(data=0x1000, numel=4, dtype=0, max_norm=1.0, out=0x2000, ws=0x3000, n=1 << 20):
        t = np.zeros(1, _SPAN_ROW)
        t["data"], t["numel"], t["dtype"] = data, numel, dtype
        return lib.tps_grad_norm(t.ctypes.data, 1, max_norm, out, ws, n, None)
    assert call(data=0) == 9 and call(numel=-1) == 1 and call(dtype=I64) == 3 and call(data=0x1001) == 4
    assert call(max_norm=math.nan) == 9 and call(out=0) == 9 and call(ws=0) == 6 and call(ws=0x3010) == 6 and call(n=16) == 6
    assert lib.tps_grad_norm_workspace_bytes(-1) == 0


def test_prepared_scalars_are_the_formulas():
    from backward_tcgen05_tma_gemms_gb300 import api
    s = api.adamw_scalars(0.25, 3, 0.5, 0.75, 0.125, seed=77)
    f = s.view(torch.float32)
    assert f[0].item() == np.float32(0.25 / (1 - 0.5 ** 3))
    assert f[1].item() == np.float32(1 / math.sqrt(1 - 0.75 ** 3))
    assert f[2].item() == np.float32(1 - 0.25 * 0.125) and s[3].item() == 77


def test_python_refusals():
    from backward_tcgen05_tma_gemms_gb300 import api
    with pytest.raises(ValueError, match="GPU"):
        api.adamw_plan([torch.zeros(3)])
    with pytest.raises(ValueError, match="GPU"):
        api.grad_norm([torch.zeros(3)])
    with pytest.raises(ValueError, match="GPU"):
        api.rope_fwd(api.rope_plan(2), torch.zeros(1, 1, 2), None, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="shape"):
        api.rope_fwd(api.rope_plan(2), torch.zeros(1, 6), None, torch.zeros(1, dtype=torch.int64), head_dim=4)
