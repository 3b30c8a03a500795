"""Head cross entropy in pieces of the vocabulary (linear_ce_fwd / _bwd)
against the formulas in float64 ("多卡张量：拆开计算，再合回同一结果", 04 /
VOCABULARY SHARDS: loss and dlogits from combined maxima and sums).

Tolerances are bounds: a logit is a sum of d products in fp32, off by at most
d 2^-23 sum |h w| (the tensor cores truncate); e^{z - lse} is then off by that
twice, relatively, and by 2^-19 for the exponential, the logarithm and the
rounded exponent; dz is rounded to bf16 for bf16 operands (half a step, 2^-8);
sums of n fp32 terms add n 2^-23, and a bf16 result 2^-8."""
import numpy as np
import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
IGN = -100


def case(seed, T, d, V, layout, dtype, ignored=0, vocab=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, d, generator=g).to(dtype)
    W = (torch.randn(d, V, generator=g) * scale / d ** 0.5 * 2).to(dtype)
    if layout == "out_in":
        W = W.t().contiguous()
    y = torch.randint(0, vocab or V, (T,), generator=g)
    y[torch.randperm(T, generator=g)[:ignored]] = IGN
    return h.cuda(), W.cuda(), y.cuda()


def reference(h, W, y, layout, reduction="none", vocab=0, up=None, denom=0.0):
    """Values and bounds of (loss, total, lse, dh, dW)."""
    T, d = h.shape
    bf16 = h.dtype == torch.bfloat16
    h, W = h.double(), (W if layout == "in_out" else W.t()).double()
    V = W.shape[1]
    n = vocab or V
    Wn = W[:, :n]
    z, mag = h @ Wn, h.abs() @ Wn.abs()
    ez = d * 2.0 ** -23 * mag.amax(1)
    lse = torch.logsumexp(z, 1)
    e_lse = ez + 2.0 ** -19 * (1 + lse.abs())
    kept = (y >= 0) & (y < n)
    yy = torch.where(kept, y, 0)[:, None].long()
    loss = torch.where(kept, lse - z.gather(1, yy)[:, 0], 0.0)
    D = 1.0
    if reduction == "mean":
        D = denom if denom > 0 else max(1, int(kept.sum()))
    g = torch.ones(T, dtype=torch.float64, device=h.device) if up is None else up.double().expand(T)
    g = torch.where(y == IGN, 0.0, g / D)[:, None]
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, yy, kept[:, None].double())
    dz = g * (p - hot)
    e_dz = g.abs() * p * (2 * ez[:, None] + 2.0 ** -19) + dz.abs() * (2.0 ** -8 if bf16 else 2.0 ** -23)
    dh, e_dh = dz @ Wn.t(), e_dz @ Wn.abs().t() + n * 2.0 ** -23 * (dz.abs() @ Wn.abs().t())
    dW, e_dW = torch.zeros(d, V).double().to(h.device), torch.zeros(d, V).double().to(h.device)
    dW[:, :n], e_dW[:, :n] = h.t() @ dz, h.abs().t() @ e_dz + T * 2.0 ** -23 * (h.abs().t() @ dz.abs())
    if layout == "out_in":
        dW, e_dW = dW.t(), e_dW.t()
    total = loss.sum() / D
    return {"loss": (loss, 2 * e_lse), "total": (total, (2 * e_lse).sum() / D + total.abs() * 2.0 ** -23),
            "lse": (lse, e_lse), "dh": (dh, e_dh), "dW": (dW, e_dW)}


def near(got, want, what):
    ref, bound = want
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound - 1e-30
    assert (over <= 0).all(), f"{what}: {over.max().item():.3e} over its bound {bound.max().item():.3e}"


def check(h, W, y, layout, reduction="none", vocab=0, denom=0.0, grad=torch.float32, piece=0, up=None):
    T, d = h.shape
    V = W.shape[1] if layout == "in_out" else W.shape[0]
    kw = dict(weight_layout=layout, ignore_index=IGN, vocab_size=vocab, reduction=reduction, denominator=denom)
    ws = None
    if piece:
        n = max(api.linear_ce_workspace_bytes(T, d, V, t, b, piece) for t in (h.dtype, torch.float32) for b in (0, 1))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    loss, total, lse = api.linear_ce_fwd(h, W, y, workspace=ws, **kw)
    dh, dW = api.linear_ce_bwd(h, W, y, lse, up, grad_dtype=grad, workspace=ws, **kw)
    assert api.last_device_error() == 0
    ref = reference(h, W, y, layout, reduction, vocab, up, denom)
    near(lse, ref["lse"], "lse")
    near(loss, ref["loss"], "loss")
    if reduction != "none":
        near(total, ref["total"], "total")
    near(dh, ref["dh"], "dHidden")
    near(dW, ref["dW"], "dWhead")
    assert not loss[y == IGN].any() and not dh[y == IGN].any()
    return loss, total, lse, dh, dW


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("T,d,V", [(1, 8, 8), (1, 64, 1000), (2, 40, 128), (31, 128, 264), (129, 72, 2056),
                                   (255, 256, 520), (257, 136, 3000), (1000, 512, 4104)])
def test_bf16_sizes(T, d, V, layout):
    check(*case(T + V, T, d, V, layout, torch.bfloat16), layout)


@pytest.mark.parametrize("V", [1, 7, 127, 129, 255, 257, 2051])
def test_bf16_odd_vocabulary(V):
    check(*case(V, 70, 96, V, "out_in", torch.bfloat16, ignored=5), "out_in", "mean")


@pytest.mark.parametrize("layout,T,d,V", [("in_out", 5, 24, 77), ("in_out", 66, 12, 801), ("out_in", 33, 10, 400)])
def test_bf16_outside_tma(layout, T, d, V):
    check(*case(3, T, d, V, layout, torch.bfloat16, ignored=2), layout, "sum", piece=256)


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("T,d,V", [(1, 1, 1), (1, 16, 300), (37, 48, 1000), (130, 65, 1537)])
def test_fp32(T, d, V, layout):
    check(*case(T, T, d, V, layout, torch.float32, ignored=T // 8), layout, "mean", piece=512)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("d,V,vocab", [(8, 16, 0), (72, 136, 129), (1000, 1288, 0), (2056, 520, 513)])
def test_few_tokens(T, d, V, vocab, layout, dtype):
    """One to eight tokens read the head once, a block for 128 columns."""
    h, W, y = case(T + d, T, d, V, layout, dtype, vocab=vocab)
    loss, total, lse = api.linear_ce_fwd(h, W, y, weight_layout=layout, vocab_size=vocab, reduction="sum")
    ref = reference(h, W, y, layout, "sum", vocab)
    near(lse, ref["lse"], "lse")
    near(loss, ref["loss"], "loss")
    near(total, ref["total"], "total")


def test_few_tokens_with_masked_and_infinite_logits():
    h, W, y = case(2, 4, 64, 300, "out_in", torch.float32)
    W[:256] = 0
    W[:256, 0] = -float("inf")  # two whole blocks of columns, and all but 44 logits, are -inf for positive h
    h = h.abs() + 0.1
    y[:] = 290
    loss, _, lse = api.linear_ce_fwd(h, W, y, weight_layout="out_in")
    want = torch.logsumexp(h.double() @ W[256:].double().t(), 1)
    assert (lse.double() - want).abs().max() <= 64 * 2.0 ** -23 * (h.double() @ W[256:].double().abs().t()).max() + 2.0 ** -17
    h[1, 3] = float("nan")
    loss, _, lse = api.linear_ce_fwd(h, W, y, weight_layout="out_in")
    assert torch.isnan(lse[1]) and torch.isfinite(lse[[0, 2, 3]]).all()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding_reductions_and_upstream(reduction, dtype):
    h, W, y = case(11, 90, 64, 1040, "in_out", dtype, ignored=13, vocab=1001)
    up = torch.randn(90 if reduction == "none" else 1, generator=torch.Generator().manual_seed(2)).cuda()
    *_, dW = check(h, W, y, "in_out", reduction, vocab=1001, up=up, piece=256)
    assert not dW[:, 1001:].any()
    if reduction == "mean":
        check(h, W, y, "in_out", reduction, vocab=1001, denom=777.0, up=up)


def test_padding_columns_are_not_read():
    h, W, y = case(12, 40, 64, 640, "in_out", torch.bfloat16, vocab=600)
    W[:, 600:] = float("nan")
    loss, _, lse = api.linear_ce_fwd(h, W, y, vocab_size=600)
    dh, dW = api.linear_ce_bwd(h, W, y, lse, vocab_size=600)
    assert all(torch.isfinite(t).all() for t in (loss, lse, dh, dW)) and not dW[:, 600:].any()


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("piece", [256, 512, 1280, 0])
def test_pieces(piece, grad):
    """Pieces of every size give the same loss bit for bit and gradients in bounds."""
    h, W, y = case(5, 300, 520, 5128, "in_out", torch.bfloat16, ignored=30)
    check(h, W, y, "in_out", "mean", grad=grad, piece=piece)


@pytest.mark.parametrize("reduction", ["sum", "mean"])
def test_a_shared_upstream_gradient_is_not_rounded_to_bf16(reduction):
    """g = 1 + 2^-9 is half a bf16 step from 1.  Rounded with the one-hot term
    it would leave the whole gradient 2^-9 off; as a factor in fp32 it leaves
    what 1 - p of the label loses, p = 1 / 8192 on average, and roundings that
    average out over 200 tokens."""
    h, W, y = case(14, 200, 64, 8192, "in_out", torch.bfloat16, scale=0.05)
    up = torch.tensor([1.0 + 2.0 ** -9], device="cuda")
    _, _, lse = api.linear_ce_fwd(h, W, y, reduction=reduction)
    dh, dW = api.linear_ce_bwd(h, W, y, lse, up, reduction=reduction)
    ref = reference(h, W, y, "in_out", reduction, up=up)
    for got, want in ((dh, ref["dh"][0]), (dW, ref["dW"][0])):
        assert abs((got.double() * want).sum() / want.square().sum() - 1).item() <= 2.0 ** -11


def test_all_ignored():
    h, W, y = case(6, 20, 64, 512, "in_out", torch.bfloat16, ignored=20)
    loss, total, _, dh, dW = check(h, W, y, "in_out", "mean")
    assert total.item() == 0 and not dW.any() and not dh.any()


def test_ignored_token_with_infinite_logits_has_no_gradient():
    h, W, y = case(7, 6, 64, 512, "in_out", torch.bfloat16)
    y[2] = IGN
    h[2] = 3e38
    loss, _, lse = api.linear_ce_fwd(h, W, y, ignore_index=IGN)
    dh, _ = api.linear_ce_bwd(h, W, y, lse, ignore_index=IGN, want_dwhead=False)
    assert loss[2].item() == 0 and not dh[2].any()
    kept = torch.arange(6, device="cuda") != 2
    assert torch.isfinite(loss[kept]).all() and torch.isfinite(dh[kept]).all()


def test_large_logits_and_rows_far_apart():
    """Rows whose logits reach hundreds: nothing overflows, p is one or nothing."""
    h, W, y = case(8, 64, 128, 1024, "in_out", torch.bfloat16, scale=60.0)
    loss, _, lse = api.linear_ce_fwd(h, W, y)
    z = h.double() @ W.double()
    want = torch.logsumexp(z, 1)
    bound = 128 * 2.0 ** -23 * (h.double().abs() @ W.double().abs()).amax(1) + 2.0 ** -19 * (1 + want.abs())
    assert ((lse.double() - want).abs() <= bound).all()
    dh, dW = api.linear_ce_bwd(h, W, y, lse)
    assert torch.isfinite(dh).all() and torch.isfinite(dW).all()


def test_bad_label_is_reported():
    h, W, y = case(9, 10, 64, 512, "in_out", torch.bfloat16)
    y[4] = 512
    loss, _, lse = api.linear_ce_fwd(h, W, y)
    assert api.last_device_error() == api.ERR_LABEL
    assert torch.isnan(loss[4]) and torch.isfinite(lse).all()
    dh, _ = api.linear_ce_bwd(h, W, y, lse, want_dwhead=False)
    assert api.last_device_error() == api.ERR_LABEL
    want = torch.softmax(h[4].double() @ W.double(), 0) @ W.double().t()  # no one-hot term
    assert torch.allclose(dh[4].double(), want, atol=2.0 ** -6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_tokens_than_one_forward_block(dtype):
    """65536 rows go through one forward GEMM; the rest follow."""
    check(*case(13, 65536 + 300, 16, 40, "in_out", dtype, ignored=1000), "in_out", "sum")


def test_empty_batch():
    h, W, y = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, 512, dtype=torch.bfloat16,
                                                                                 device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    loss, total, lse = api.linear_ce_fwd(h, W, y, reduction="mean")
    dh, dW = api.linear_ce_bwd(h, W, y, lse, reduction="mean")
    assert loss.numel() == 0 and total.item() == 0 and dh.shape == (0, 64) and not dW.any()


def test_strided_views_int32_labels_and_another_stream():
    g = torch.Generator().manual_seed(1)
    big = torch.randn(50, 200, generator=g).to(torch.bfloat16).cuda()
    h = big[:, 8:136]                                            # rows 400 bytes apart
    W = (torch.randn(600, 256, generator=g) * 0.1).to(torch.bfloat16).cuda()[:, 64:192]  # out_in, strided
    y = torch.randint(0, 600, (50,), generator=g).cuda()
    out = torch.full((50, 160), 7.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss, _, lse = api.linear_ce_fwd(h, W, y.to(torch.int32), weight_layout="out_in")
        dW = torch.empty(600, 128, device="cuda")
        dh, dW = api.linear_ce_bwd(h, W, y.to(torch.int32), lse, weight_layout="out_in", out=(out[:, 16:144], dW))
    s.synchronize()
    ref = reference(h, W, y, "out_in")
    near(loss, ref["loss"], "loss")
    near(dh, ref["dh"], "dHidden")
    near(dW, ref["dW"], "dWhead")
    assert (out[:, :16] == 7).all() and (out[:, 144:] == 7).all()


def test_transposed_weight_and_gradient_outputs():
    """A d x V view of V x d storage (no copy), and dWhead written the same way."""
    h, W, y = case(21, 60, 64, 704, "out_in", torch.bfloat16)
    loss, _, lse = api.linear_ce_fwd(h, W.t(), y)
    store = torch.empty(704, 64, device="cuda")
    dh, dW = api.linear_ce_bwd(h, W.t(), y, lse, out=(torch.empty(60, 64, device="cuda"), store.t()))
    ref = reference(h, W, y, "out_in")
    near(loss, ref["loss"], "loss")
    near(dh, ref["dh"], "dHidden")
    near(store, ref["dW"], "dWhead")


def test_gradient_is_the_difference_quotient():
    """fp32: d(sum of losses)/dW and /dh against central differences in float64 of the formula."""
    h, W, y = case(31, 9, 12, 40, "in_out", torch.float32)
    _, _, lse = api.linear_ce_fwd(h, W, y)
    dh, dW = api.linear_ce_bwd(h, W, y, lse)

    def total(hh, ww):
        z = hh @ ww
        return (torch.logsumexp(z, 1) - z.gather(1, y[:, None])[:, 0]).sum()
    hd, Wd, e = h.double(), W.double(), 1e-5
    for i, j in ((0, 0), (3, 17), (11, 39)):
        t = torch.zeros_like(Wd)
        t[i, j] = e
        assert abs(((total(hd, Wd + t) - total(hd, Wd - t)) / (2 * e) - dW[i, j]).item()) < 1e-4
    for i, j in ((0, 0), (4, 5), (8, 11)):
        t = torch.zeros_like(hd)
        t[i, j] = e
        assert abs(((total(hd + t, Wd) - total(hd - t, Wd)) / (2 * e) - dh[i, j]).item()) < 1e-4


def test_matches_the_operator_that_keeps_logits():
    h, W, y = case(41, 260, 256, 2048, "in_out", torch.bfloat16, ignored=20)
    loss, _, lse = api.linear_ce_fwd(h, W, y, ignore_index=IGN)
    dh, dW = api.linear_ce_bwd(h, W, y, lse, ignore_index=IGN)
    loss2, _, _, dh2, dW2, _ = api.vocab_ce_fwd_bwd_ex(h, W, y, 4, ignore_index=IGN, want_dwhead=True)
    for a, b in ((loss, loss2), (dh, dh2), (dW, dW2)):
        assert (a - b).norm() <= 5e-3 * b.norm()


def test_same_bits_every_time_and_in_a_graph():
    h, W, y = case(51, 512, 512, 4096, "in_out", torch.bfloat16, ignored=9)
    kw = dict(ignore_index=IGN, reduction="mean")
    first = None
    for _ in range(3):
        loss, total, lse = api.linear_ce_fwd(h, W, y, **kw)
        dh, dW = api.linear_ce_bwd(h, W, y, lse, **kw)
        now = [t.clone() for t in (loss, total, lse, dh, dW)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    ws = torch.empty(api.linear_ce_workspace_bytes(512, 512, 4096, torch.bfloat16, True), dtype=torch.uint8, device="cuda")
    out, grads = [torch.zeros_like(t) for t in first[:3]], [torch.zeros_like(t) for t in first[3:]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.linear_ce_fwd(h, W, y, workspace=ws, out=out, **kw)
        api.linear_ce_bwd(h, W, y, out[2], workspace=ws, out=grads, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out + grads))


def test_debug_free_of_stray_writes():
    """Guard bands around every output stay untouched (odd sizes, several pieces)."""
    h, W, y = case(61, 77, 72, 1031, "out_in", torch.bfloat16)
    T, d, V = 77, 72, 1031
    need = api.linear_ce_workspace_bytes(T, d, V, torch.bfloat16, True, 256)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")

    def guarded(n):
        t = torch.full((n + 128,), 9.0, device="cuda")
        return t, t[64:64 + n]
    big_l, loss = guarded(T)
    big_s, lse = guarded(T)
    big_h, dh = guarded(T * d)
    big_w, dW = guarded(V * d)
    api.linear_ce_fwd(h, W, y, weight_layout="out_in", workspace=ws, out=(loss, None, lse))
    api.linear_ce_bwd(h, W, y, lse, weight_layout="out_in", workspace=ws[:need], out=(dh.view(T, d), dW.view(V, d)))
    torch.cuda.synchronize()
    for t in (big_l, big_s, big_h, big_w):
        assert (t[:64] == 9).all() and (t[-64:] == 9).all()
    assert (ws[need:] == 0xA5).all()
