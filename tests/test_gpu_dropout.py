"""Dropout against its mask from the published generator, bit for bit where the
result is a product alone, else within one rounding an operation."""
import math

import pytest
import torch

import philox_plain
from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def mask(shape, p, seed, site):
    return torch.from_numpy(philox_plain.mask(shape, p, seed, site)).cuda()


@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (5, 3), (3, 8), (100, 77), (64, 512), (2, 3, 40), (1, 20000)])
@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_values(shape, t, p):
    x = torch.randn(shape, device="cuda").to(t)
    res = torch.randn(shape, device="cuda").to(t)
    seed, site = 0x123456789abcdef0, 5
    m = mask(shape, p, seed, site)
    scale = m.float()
    y = api.dropout_fwd(x, p, seed, site=site)
    if p:
        assert torch.equal(y, (x.float() * scale).to(t))
        assert torch.equal(api.dropout_bwd(x, p, seed, site=site), y)
    else:
        assert torch.equal(y, x)
    z = api.dropout_fwd(x, p, seed, site=site, residual=res).double()
    want = x.double() * (m if p else 1.0) + res.double()
    lim = torch.finfo(t).eps / 2 * want.abs() + 2 * U * (x.double().abs() * 2 + res.double().abs())
    assert ((z - want).abs() <= lim).all()


@pytest.mark.parametrize("extra,shift", [(8, 8), (8, 3), (5, 0)])
@pytest.mark.parametrize("d", [64, 77])
def test_pitched_rows(extra, shift, d):
    big = torch.randn(20, d + extra, device="cuda").to(BF)
    x = big[:, shift:shift + d]
    y = api.dropout_fwd(x, 0.3, 9)
    assert torch.equal(y, (x.float() * mask((20, d), 0.3, 9, 0).float()).to(BF))
    out = torch.full((20, d + extra), 3.0, device="cuda").to(BF)
    api.dropout_fwd(x, 0.3, 9, out=out[:, shift:shift + d])
    assert torch.equal(out[:, shift:shift + d], y)
    assert (out[:, :shift] == 3).all() and (out[:, shift + d:] == 3).all()


def test_unaligned_flat():
    x = torch.randn(1001, device="cuda")[1:]
    assert torch.equal(api.dropout_fwd(x, 0.5, 3), x * mask((1000,), 0.5, 3, 0).float())


@pytest.mark.parametrize("xt,rt,yt", [(a, b, c) for a in (BF, FP) for b in (BF, FP) for c in (BF, FP)])
def test_mixed_types(xt, rt, yt):
    x, res = torch.randn(30, 40, device="cuda").to(xt), torch.randn(30, 40, device="cuda").to(rt)
    y = api.dropout_fwd(x, 0.25, 4, residual=res, out=torch.empty(30, 40, dtype=yt, device="cuda")).double()
    want = x.double() * mask((30, 40), 0.25, 4, 0) + res.double()
    lim = torch.finfo(yt).eps / 2 * want.abs() + 2 * U * (x.double().abs() * 2 + res.double().abs())
    assert ((y - want).abs() <= lim).all()


def test_in_place_and_dropped_not_finite():
    x = torch.randn(50, 64, device="cuda")
    want = api.dropout_fwd(x, 0.5, 1, residual=x)
    a = x.clone()
    api.dropout_fwd(a, 0.5, 1, residual=a, out=a)
    assert torch.equal(a, want)
    m = mask((50, 64), 0.5, 1, 0) > 0
    x.fill_(math.nan)
    y = api.dropout_fwd(x, 0.5, 1)
    assert torch.isnan(y[m]).all() and (y[~m] == 0).all()


def test_share_and_independence():
    """2^22 draws: the share kept within five deviations; seeds and sites agree as often as chance has it."""
    n, p = 1 << 22, 0.1
    x = torch.ones(n, device="cuda")
    masks = [api.dropout_fwd(x, p, s, site=i) > 0 for s, i in ((1, 0), (2, 0), (1, 1), (1 << 32, 0))]
    for m in masks:
        assert abs(m.double().mean().item() - (1 - 6554 / 65536)) <= 5 * math.sqrt(p * (1 - p) / n)
    same = p * p + (1 - p) * (1 - p)
    for i in range(4):
        for j in range(i):
            agree = (masks[i] == masks[j]).double().mean().item()
            assert abs(agree - same) <= 5 * math.sqrt(same * (1 - same) / n) + 1e-4


def test_seed_on_the_gpu():
    x = torch.randn(64, 64, device="cuda")
    for s in (0, 5, -1, 2 ** 62 + 3):
        assert torch.equal(api.dropout_fwd(x, 0.5, torch.tensor([s], device="cuda")), api.dropout_fwd(x, 0.5, s))
    with pytest.raises(ValueError, match="GPU"):
        api.dropout_fwd(x, 0.5, torch.tensor([1]))


def test_empty_and_refused():
    assert api.dropout_fwd(torch.empty(0, 8, device="cuda"), 0.5, 1).shape == (0, 8)
    x = torch.randn(4, 8, device="cuda")
    for p in (-0.5, 1.5, math.nan):
        with pytest.raises(api.TpsError) as e:
            api.dropout_fwd(x, p, 1)
        assert e.value.code == api.ERR_ARG
    with pytest.raises(ValueError, match="shape"):
        api.dropout_fwd(x, 0.5, 1, residual=torch.randn(4, 9, device="cuda"))
