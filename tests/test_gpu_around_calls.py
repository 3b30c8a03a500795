"""What a call of norm, dropout, e4m3 rows and the linear product does beside its
results: the memory it takes, and what autograd is told of tensors it writes."""
import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("T", [1, 5, 8])
def test_few_fp32_rows_take_no_workspace(T, layout):
    """Nothing but the output is allocated, where laying W out would take six bytes an element; a W that
    does not start on 16 bytes still goes that way."""
    K, N = 1024, 2048
    shape = (K, N) if layout == "in_out" else (N, K)
    x, W = torch.randn(T, K, device="cuda"), torch.randn(*shape, device="cuda")
    off = torch.empty(K * N + 1, device="cuda")[1:].view(*shape)
    off.copy_(W)
    api.linear_fwd(x, W, weight_layout=layout)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y, _ = api.linear_fwd(x, W, weight_layout=layout)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 20
    z, _ = api.linear_fwd(x, off, weight_layout=layout)
    assert torch.cuda.max_memory_allocated() - before >= 6 * K * N
    w64 = W.double() if layout == "in_out" else W.double().t()
    want, S = x.double() @ w64, x.double().abs() @ w64.abs()
    for got in (y, z):  # sums of K products, each rounding at most 2^-24 of what is summed, and the output's
        assert ((got.double() - want).abs() <= (K + 2) * 2.0 ** -24 * S).all()


def calls():
    """name -> (call, outputs it is given)."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g).to(BF)
    x, res, dy, W, z = r(16, 64), r(16, 64), r(16, 64), r(64, 64), r(16, 64)
    rstd, dw, vec = torch.ones(16, device="cuda"), torch.empty(64, device="cuda"), torch.empty(16, device="cuda")
    q8, y8 = (torch.empty(16, 64, device="cuda", dtype=torch.float8_e4m3fn) for _ in range(2))
    out = {}
    y, h = r(16, 64), r(16, 64)
    out["norm"] = (lambda: api.rmsnorm_fwd(x, residual=res, out=(y, None, h, rstd)), [y, h, rstd])
    over, r2 = r(16, 64), torch.ones(16, device="cuda")
    out["norm over its input"] = (lambda: api.rmsnorm_fwd(over, out=(over, None, None, r2)), [over, r2])
    joined, y2, r3 = r(16, 64), r(16, 64), torch.ones(16, device="cuda")
    out["norm over the residual"] = (lambda: api.rmsnorm_fwd(x, residual=joined, out=(y2, None, joined, r3)), [joined, y2, r3])
    r4, s4 = torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    out["norm to e4m3"] = (lambda: api.rmsnorm_fwd(x, out_dtype=y8.dtype, out=(y8, s4, None, r4)), [y8, s4, r4])
    dx, ds = r(16, 64), r(16, 64)
    out["norm backward"] = (lambda: api.rmsnorm_bwd(dy, x, None, vec.fill_(1.0), out=(dx, ds, dw)), [dx, ds, dw])
    d1, d2 = r(16, 64), r(16, 64)
    out["dropout"] = (lambda: api.dropout_fwd(d1, 0.5, 3, out=d1), [d1])
    out["dropout backward"] = (lambda: api.dropout_bwd(dy, 0.5, 3, out=d2), [d2])
    sq = torch.empty(16, device="cuda")
    out["e4m3 rows"] = (lambda: api.quantize_e4m3(x, out=(q8, sq)), [q8, sq])
    l1, l2 = r(16, 64), r(16, 64)
    out["linear"] = (lambda: api.linear_fwd(x, W, act="silu", out=(l1, l2)), [l1, l2])
    l3 = r(16, 64)
    out["linear over the residual"] = (lambda: api.linear_fwd(x, W, residual=l3, out=(l3, None)), [l3])
    g1, g2, g3 = r(16, 64), r(64, 64), torch.empty(64, device="cuda")
    out["linear backward"] = (lambda: api.linear_bwd(x, W, dy, pre=z, act="silu", out=(g1, g2, g3)), [g1, g2, g3])
    return out


def test_writes_are_counted():
    """Each tensor that a call was given as an output has another version afterwards, the inputs the same."""
    for name, (call, given) in calls().items():
        before = [t._version for t in given]
        call()
        assert all(t._version > v for t, v in zip(given, before)), name
    x = torch.randn(16, 64, device="cuda")
    y, _, _, rstd = api.rmsnorm_fwd(x)
    api.linear_fwd(x, torch.randn(64, 64, device="cuda"))
    assert x._version == 0 and y._version == 0 and rstd._version == 0


def test_a_refused_call_counts_nothing():
    x, y = torch.randn(4, 64, device="cuda"), torch.randn(4, 63, device="cuda")
    before = y._version
    with pytest.raises(ValueError, match="shape"):
        api.dropout_fwd(x, 0.5, 1, out=y)
    assert y._version == before


def test_an_eager_graph_notices():
    """exp saves its result for its backward pass, which raises once a call has written over it."""
    for call in (lambda s: api.rmsnorm_fwd(s, out=(s, None, None, torch.empty(8, device="cuda"))),
                 lambda s: api.dropout_fwd(s, 0.5, 1, out=s),
                 lambda s: api.linear_fwd(torch.randn(8, 64, device="cuda"), torch.randn(64, 64, device="cuda"), residual=s,
                                          out=(s, None)),
                 lambda s: api.rmsnorm_bwd(s, s.clone(), None, torch.ones(8, device="cuda"), out=(s, None, None))):
        leaf = torch.randn(8, 64, device="cuda", requires_grad=True)
        saved = leaf.exp()
        call(saved.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.sum().backward()


def test_inference_tensors():
    with torch.inference_mode():
        x = torch.randn(8, 64, device="cuda")
        want = api.dropout_fwd(x, 0.5, 1)
        api.dropout_fwd(x, 0.5, 1, out=x)
    assert torch.equal(x, want)
    api.dropout_fwd(torch.zeros(8, 64, device="cuda"), 0.5, 1, out=x)
    assert not x.any()


def test_writes_of_the_other_calls_are_counted():
    g = torch.Generator(device="cuda").manual_seed(2)

    def r(*s, t=FP):
        return torch.randn(*s, device="cuda", generator=g).to(t)
    T, d, F, V = 32, 64, 128, 256
    X, W1, W2, GY, h = r(T, d, t=BF), r(d, F, t=BF), r(F, d, t=BF), r(T, d, t=BF), r(T, d, t=BF)
    Wh, labels = r(d, V, t=BF), torch.randint(0, V, (T,), device="cuda", generator=g)
    q, k, pos = r(T, 2, 32, t=BF), r(T, 1, 32, t=BF), torch.arange(T, device="cuda")
    plan = api.rope_plan(32)
    lse = api.linear_ce_fwd(h, Wh, labels)[2]
    cases = {
        "matmul": (lambda out: api.matmul_fwd_bwd(X, W1, r(T, F, t=BF), 2, "rows", out=out), [r(T, F), r(T, d), r(d, F)]),
        "mlp": (lambda out: api.mlp_fwd_bwd(X, W1, W2, GY, 2, out=out), [r(T, d), r(T, d), r(d, F), r(F, d)]),
        "mlp without workspace": (lambda out: api.mlp_fwd_bwd_noalloc(X, W1, W2, GY, 2, out=out), [r(T, d), r(T, d), r(d, F), r(F, d)]),
        "gated mlp": (lambda out: api.glu_mlp_fwd_bwd(X, W1, W1, W2, GY, 2, out=out), [r(T, d), r(T, d), r(d, F), r(d, F), r(F, d)]),
        "cross entropy": (lambda out: api.vocab_ce_fwd_bwd(h, Wh, labels, 2, out=out),
                          [r(T), r(T, V, t=BF), r(T, d), torch.zeros(T, device="cuda", dtype=torch.int32)]),
        "head cross entropy": (lambda out: api.linear_ce_fwd(h, Wh, labels, out=out), [r(T), None, r(T)]),
        "its backward": (lambda out: api.linear_ce_bwd(h, Wh, labels, lse, out=out), [r(T, d), r(d, V)]),
        "rope": (lambda out: api.rope_fwd(plan, *out, pos, out=out), [q, k]),
        "rope backward": (lambda out: api.rope_bwd(plan, *out, pos, out=out), [q, k]),
        "norm of gradients": (lambda out: api.grad_norm([X], 1.0, out=out[0]), [r(2)]),
    }
    for name, (call, out) in cases.items():
        given = [t for t in out if t is not None]
        before = [t._version for t in given]
        call(out)
        assert all(t._version > v for t, v in zip(given, before)), name


def test_last_tokens_of_a_batch():
    """Views [:, -1:] of (batch, tokens, d), in and out: as their contiguous copies."""
    big, bres, bout = (torch.randn(5, 3, 64, device="cuda").to(BF) for _ in range(3))
    x, res = big[:, -1:], bres[:, -1:]
    W = torch.randn(64, 72, device="cuda").to(BF)
    want = api.rmsnorm_fwd(x.contiguous(), residual=res.contiguous())
    got = api.rmsnorm_fwd(x, residual=res)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
    rest = bout[:, :2].clone()
    api.rmsnorm_fwd(x, residual=res, out=(bout[:, -1:], None, got[2], got[3]))
    assert torch.equal(bout[:, -1:], want[0]) and torch.equal(bout[:, :2], rest)
    assert torch.equal(api.linear_fwd(x, W)[0], api.linear_fwd(x.contiguous(), W)[0])
    assert torch.equal(api.dropout_fwd(x, 0.5, 3), api.dropout_fwd(x.contiguous(), 0.5, 3))
    assert all(torch.equal(a, b) for a, b in zip(api.quantize_e4m3(x), api.quantize_e4m3(x.contiguous())))
    a = api.rmsnorm_bwd(x, got[2], None, got[3], dh=res)
    b = api.rmsnorm_bwd(x.contiguous(), got[2], None, got[3], dh=res.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,d", [(40, 512), (700, 2048), (33, 77), (9, 20000)])
def test_sums_right_behind_their_parts(T, d, captured):
    """The kernel that adds up a gradient's parts is started before the one that writes them ends: through one
    workspace, call after call, each sum is that of its own parts, as with a wait after each call."""
    g = torch.Generator(device="cuda").manual_seed(d)
    xs = [torch.randn(T, d, device="cuda", generator=g).to(BF) for _ in range(8)]
    rstd, W = torch.ones(T, device="cuda"), torch.randn(d, 64, device="cuda", generator=g).to(BF)
    N = 64
    dys = [x[:, :N] if d % 8 == 0 else x[:, :N].contiguous() for x in xs]
    ws = torch.empty(max(api.rmsnorm_workspace_bytes(T, d), api.linear_workspace_bytes(T, d, N, FP, True)), dtype=torch.uint8,
                     device="cuda")

    def chain(wait):
        out = []
        for i, (x, dy) in enumerate(zip(xs, dys)):
            out.append(api.rmsnorm_bwd(x, xs[i - 1], None, rstd, workspace=ws)[2])
            wait()
            out.append(api.linear_bwd(x, W, dy, want_dx=False, want_dw=False, workspace=ws)[2])
            wait()
        return out
    want = chain(torch.cuda.synchronize)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(lambda: None)
        graph.replay()
    else:
        got = chain(lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    terms = xs[0].double() * xs[-1].double()  # exact in fp32: T - 1 additions, each off by at most 2^-24 of all of them
    assert ((want[0].double() - terms.sum(0)).abs() <= T * 2.0 ** -24 * terms.abs().sum(0)).all()


@pytest.mark.parametrize("T", [1, 5, 64, 300])
@pytest.mark.parametrize("K,N", [(1, 1), (50, 1), (50, 40), (130, 129)])
def test_e4m3_rows_of_any_length(T, K, N):
    """Rows that start on 16 bytes, whatever their length: what lies behind them (NaN here) is not read, and a
    single row starts where it starts.  Sums in fp32 of K products, exact ones: K 2^-24 of their magnitudes, three
    roundings of the scales and one of the output beside it."""
    E8 = torch.float8_e4m3fn

    def rows(n):
        big = torch.full((n, -(-K // 16) * 16 + 16), float("nan"), device="cuda").to(E8)
        v, scale = big[:, :K], torch.empty(n, device="cuda")
        api.quantize_e4m3(torch.randn(n, K, device="cuda"), out=(v, scale))
        return v, scale
    (x, xs), (W, ws) = rows(T), rows(N)
    y, _ = api.linear_fwd(x, W, x_scale=xs, w_scale=ws, weight_layout="out_in", out_dtype=FP)
    a, b = x.double() * xs.double()[:, None], W.double() * ws.double()[:, None]
    assert ((y.double() - a @ b.t()).abs() <= (K + 4) * 2.0 ** -24 * (a.abs() @ b.abs().t())).all()
    assert api.last_device_error() == 0
