"""Head cross entropy (linear_ce_fwd / _bwd) where it can go wrong beside the
sizes: infinite and missing logits.  Tolerances as in test_gpu_linear_ce.py."""
import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api
from test_gpu_linear_ce import IGN, case, check, near, reference

pytestmark = pytest.mark.gpu


def lse_bound(h, W, lse):
    """Of finite logits: d products in fp32, and the exponentials' 2^-19."""
    return h.shape[1] * 2.0 ** -23 * (h.double().abs() @ W.double().abs().t()).amax(1) + 2.0 ** -19 * (1 + lse.abs())


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("T,d,off", [(1, 64, 0), (8, 64, 0), (9, 64, 0), (16, 600, 0), (300, 72, 0), (3, 64, 1), (5, 4096, 0)])
def test_masked_vocabulary_entries_in_fp32(T, d, off, layout):
    """-inf in a head entry that meets positive h makes its logit -inf and
    leaves the row finite, whatever T, alignment or layout; so does +inf that
    meets negative h.  The masked columns have no gradient."""
    h, W, y = case(T + d, T, d, 301, "out_in", torch.float32)
    h[:, 2], h[:, 3] = h[:, 2].abs() + 0.1, -h[:, 3].abs() - 0.1
    W[:140, 2] = -float("inf")  # a whole tile of 128 columns and part of the next
    W[170:180, 3] = float("inf")
    kept = torch.ones(301, dtype=torch.bool, device="cuda")
    kept[:140] = kept[170:180] = False
    y = torch.where(kept[y], y, 200)
    head = torch.zeros(301 * d + 4, device="cuda")[off:off + 301 * d].view(301, d)
    head.copy_(W)
    if layout == "in_out":
        store = torch.zeros(301 * d + 4, device="cuda")[off:off + 301 * d].view(d, 301)
        head = store.copy_(W.t())
    loss, _, lse = api.linear_ce_fwd(h, head, y, weight_layout=layout)
    want = torch.logsumexp(h.double() @ W[kept].double().t(), 1)
    bound = lse_bound(h, W[kept], want)
    assert ((lse.double() - want).abs() <= bound).all()
    label = (h.double() * W[y].double()).sum(1)
    assert ((loss.double() - (want - label)).abs() <= 2 * bound).all()
    _, dW = api.linear_ce_bwd(h, head, y, lse, weight_layout=layout, want_dhidden=False)
    dW = dW if layout == "out_in" else dW.t()
    ref = reference(h, W[kept], kept.cumsum(0)[y] - 1, "out_in")["dW"]
    near(dW[kept], ref, "dWhead")
    assert not dW[~kept].any()
    assert api.last_device_error() == 0


@pytest.mark.parametrize("T", [4, 40])
def test_infinite_and_missing_logits_follow_fp32(T):
    """A row's logits are what fp32 products give: +inf, NaN for inf - inf, and NaN for a NaN in h or the head."""
    h, W, _ = case(5, T, 64, 40, "out_in", torch.float32)
    h = h.abs() + 0.1
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    W[7, 3] = float("inf")
    _, _, lse = api.linear_ce_fwd(h, W, y, weight_layout="out_in")
    assert not torch.isfinite(lse).any() and not (lse == -float("inf")).any()
    W[7, 4] = -float("inf")
    assert torch.isnan(api.linear_ce_fwd(h, W, y, weight_layout="out_in")[2]).all()
    W[7, 3:5] = 1.0
    h[2, 5] = float("inf")
    h[1, 0] = float("nan")
    _, _, lse = api.linear_ce_fwd(h, W, y, weight_layout="out_in")
    assert torch.isnan(lse[1]) and not torch.isfinite(lse[2])
    rest = [i for i in range(T) if i not in (1, 2)]
    assert torch.isfinite(lse[rest]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [2, 40])
def test_a_nan_among_masked_logits_is_not_lost(T, dtype):
    """Where everything before it in the row is -inf, a NaN still makes the row's sum NaN."""
    h, W, _ = case(6, T, 64, 400, "out_in", dtype)
    h = h.abs() + 0.1
    W[:200, 2] = -float("inf")
    W[133, 2] = float("nan")
    y = torch.full((T,), 390, device="cuda")
    loss, _, lse = api.linear_ce_fwd(h, W, y, weight_layout="out_in")
    assert torch.isnan(lse).all() and torch.isnan(loss).all()


@pytest.mark.parametrize("scale", [1.0, 1e-6, 1e20])
def test_a_gradient_that_all_tokens_share_is_not_rounded_to_bf16(scale):
    """The mean of the tokens' losses taken outside sends the same gradient to each of them (and here nothing usable to
    the ignored ones).  c = 1 + 2^-9 times a scale is up to half a bf16 step from what bf16 holds; as a factor in fp32
    it leaves what 1 - p of the label loses (p = 1 / 8192 on average) and roundings that average out over 170 tokens."""
    h, W, y = case(14, 200, 64, 8192, "in_out", torch.bfloat16, scale=0.05)
    y[::7] = IGN
    up = torch.full((200,), 1.0 + 2.0 ** -9, device="cuda") * scale
    _, _, lse = api.linear_ce_fwd(h, W, y, ignore_index=IGN)
    ref = reference(h, W, y, "in_out", up=up)
    up[::7] = float("nan")
    dh, dW = api.linear_ce_bwd(h, W, y, lse, up, ignore_index=IGN)
    for got, want in ((dh, ref["dh"][0]), (dW, ref["dW"][0])):
        assert abs((got.double() * want).sum() / want.square().sum() - 1).item() <= 2.0 ** -11
    assert not dh[::7].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_gradient_that_is_not_finite_stays_with_its_token(bad, dtype):
    h, W, y = case(15, 40, 64, 520, "in_out", dtype)
    up = torch.randn(40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 1e-3
    up[5], up[9] = bad, 0.0
    y[7] = IGN
    _, _, lse = api.linear_ce_fwd(h, W, y, ignore_index=IGN)
    dh, _ = api.linear_ce_bwd(h, W, y, lse, up, ignore_index=IGN, want_dwhead=False)
    rest = torch.arange(40, device="cuda") != 5
    want, bound = reference(h, W, y, "in_out", up=torch.nan_to_num(up, 0.0, 0.0))["dh"]
    near(dh[rest], (want[rest], bound[rest]), "dHidden")
    assert not torch.isfinite(dh[5]).any() and not dh[7].any() and not dh[9].any()
    for reduction in ("sum", "mean"):
        dh, _ = api.linear_ce_bwd(h, W, y, lse, torch.tensor([bad], device="cuda"), ignore_index=IGN, reduction=reduction)
        assert not dh[7].any() and not torch.isfinite(dh[rest.logical_and(torch.arange(40, device="cuda") != 7)]).any()


def test_no_gradient_at_all():
    h, W, y = case(16, 40, 64, 520, "in_out", torch.bfloat16)
    _, _, lse = api.linear_ce_fwd(h, W, y)
    for up, reduction in ((torch.zeros(40, device="cuda"), "none"), (torch.zeros(1, device="cuda"), "sum")):
        dh, dW = api.linear_ce_bwd(h, W, y, lse, up, reduction=reduction)
        assert not dh.any() and not dW.any()


def test_fp32_gradients_of_rows_with_a_large_lse():
    """z and lse near 1000 that fp32 holds exactly: e^{z - lse} is off by the hardware exponential's 2^-22 and two
    roundings of the difference's at most 8 binary digits of exponent, 2^-20 together, not by lse's own magnitude."""
    z = 1000 + 37.0 * torch.arange(8)[:, None] + torch.arange(64)[None] / 64.0
    y = torch.arange(8) * 7
    lse = torch.logsumexp(z.double(), 1).float()
    _, dW = api.linear_ce_bwd(torch.eye(8).cuda(), z.cuda(), y.cuda(), lse.cuda(), want_dhidden=False)
    p = torch.exp(z.double() - lse.double()[:, None])
    want = p - torch.zeros_like(p).scatter_(1, y[:, None], 1.0)
    assert ((dW.cpu().double() - want).abs() <= 2.0 ** -20 * p + 2.0 ** -23 * want.abs()).all()


def test_workspaces_that_are_refused():
    h, W, y = case(17, 20, 64, 520, "in_out", torch.bfloat16)
    shared = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24)
    with pytest.raises(api.TpsError, match="contiguous"):
        api.linear_ce_fwd(h, W, y, workspace=shared)
    with pytest.raises(api.TpsError, match="contiguous"):
        api.grad_norm([h], workspace=shared)
    with pytest.raises(ValueError, match="GPU"):
        api.linear_ce_fwd(h, W, y, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        api.grad_norm([h], workspace=torch.empty(1 << 24, dtype=torch.uint8))


@pytest.mark.parametrize("split", ["01", "03", "11", "13", "116"])
@pytest.mark.parametrize("reduction,dtype,grad", [("mean", torch.bfloat16, torch.float32), ("sum", torch.bfloat16, torch.bfloat16),
                                                  ("none", torch.bfloat16, torch.float32), ("mean", torch.float32, torch.float32)])
@pytest.mark.parametrize("T,d,V", [(300, 520, 1300), (70, 1032, 4100)])
def test_every_way_to_sum_dhidden(T, d, V, reduction, dtype, grad, split, monkeypatch):
    """dHidden on 256 x 256 and 256 x 512 tiles, in one and in several K runs, over pieces of 1024 columns and over one
    piece, with an upstream gradient: the paths that large shapes take by themselves."""
    monkeypatch.setenv("TPS_LCE_SPLIT", split)
    for layout, piece in (("out_in", 1024), ("out_in", 0), ("in_out", 1024)):
        V8 = V if layout == "out_in" else V - V % 8
        h, W, y = case(T, T, d, V8, layout, dtype, ignored=T // 10)
        up = torch.randn(T if reduction == "none" else 1, generator=torch.Generator().manual_seed(2)).cuda()
        check(h, W, y, layout, reduction, grad=grad, piece=piece, up=up)


@pytest.mark.parametrize("layout,T,d,V,dtype", [("out_in", 90, 72, 1031, torch.float32), ("in_out", 300, 40, 1027, torch.bfloat16),
                                                ("in_out", 20, 64, 2000, torch.float32)])
def test_pieces_leave_the_loss_as_it_is(layout, T, d, V, dtype):
    """Operands that are laid out go piece by piece in the forward pass too: loss and lse are the same bits whatever the
    piece, dWhead as well, and dHidden within the bounds."""
    h, W, y = case(7, T, d, V, layout, dtype, ignored=3)
    first = None
    for piece in (256, 512, 1024, 0):
        loss, _, lse, _, dW = check(h, W, y, layout, piece=piece)
        first = first or (loss, lse, dW)
        assert all(torch.equal(a, b) for a, b in zip(first, (loss, lse, dW)))


@pytest.mark.parametrize("d", [4096, 32768])
def test_long_fp32_sums_keep_their_precision(d):
    """One vocabulary entry: lse is the logit, a sum of d positive products.  Tensor cores cut a partial sum at each
    step of 16 products, at worst one 2^-23 of it, for 32 steps into an accumulator; the d / 512 accumulators are added
    with 2^-24 each.  (One accumulator throughout would be off by about 2^-24 for each of d / 16 steps: 1e-4 at 32768.)"""
    g = torch.Generator().manual_seed(1)
    h, W = torch.rand(16, d, generator=g).cuda(), torch.rand(1, d, generator=g).cuda()
    _, _, lse = api.linear_ce_fwd(h, W, torch.zeros(16, dtype=torch.int64, device="cuda"), weight_layout="out_in")
    want = h.double() @ W[0].double()
    assert ((lse.double() - want).abs() <= (32 * 2.0 ** -23 + (d / 512 + 4) * 2.0 ** -24) * want).all()
