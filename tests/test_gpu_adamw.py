"""AdamW over many tensors and the gradient norm, against the update in
float64.

Bounds for fp32 moments: m and v are a sum of two products of rounded
constants, 6 and 8 roundings of 2^-24 of the terms' magnitudes; the step adds
the square root, the division and their operands (8 roundings), the weight
two products and a difference.  e4m3 moments are checked to be one of the two
e4m3 neighbours of their value over the block's scale, nearest (half a step)
or at random with the right expectation."""
import math

import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
E4M3 = torch.float8_e4m3fn
GRID = torch.arange(127, dtype=torch.uint8).view(E4M3).double()  # the non-negative numbers, ascending


def tensors(sizes, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dtype).cuda() for n in sizes]


def moments(plan, i):
    """(m, v) of tensor i in float64."""
    m, v = plan.m[i], plan.v[i]
    if m.dtype == E4M3:
        n = m.numel()
        e = lambda s: s.double().repeat_interleave(256)[:n]  # noqa: E731
        return m.float().double() * e(plan.m_scale[i]), (v.float().double() * e(plan.v_scale[i])) ** 2
    return m.double(), v.double()


def formula(w, g, m, v, step, coef=1.0, lr=0.0, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0):
    g = g.double() * coef
    m2 = beta1 * m + (1 - beta1) * g
    v2 = beta2 * v + (1 - beta2) * g * g
    em = 6 * U * (beta1 * m.abs() + (1 - beta1) * g.abs())
    den = (v2 / (1 - beta2 ** step)).sqrt() + eps
    u = lr / (1 - beta1 ** step) * m2 / den
    eu = lr / (1 - beta1 ** step) * em / den + u.abs() * 16 * U
    w2 = w.double() * (1 - lr * weight_decay) - u
    return w2, eu + 4 * U * (w.double().abs() + w2.abs()), m2, em, v2, 8 * U * v2


@pytest.mark.parametrize("param,master,grad", [(torch.float32, False, torch.float32), (torch.float32, False, torch.bfloat16),
                                               (torch.bfloat16, True, torch.bfloat16), (torch.bfloat16, True, torch.float32),
                                               (torch.bfloat16, False, torch.bfloat16), (torch.bfloat16, False, torch.float32)])
@pytest.mark.parametrize("sizes", [[1], [256], [255, 0, 257, 4096, 3, 100003], [5] * 340])
def test_fp32_moments(sizes, param, master, grad):
    ps = tensors(sizes, param, 1)
    plan = api.adamw_plan(ps, master=master)
    for step in (1, 2, 3):
        gs = tensors(sizes, grad, 10 + step, 0.1)
        before = [((plan.master[i] if master else p).clone(), *moments(plan, i)) for i, p in enumerate(ps)]
        api.adamw_step(plan, gs, step=step, **HP)
        for i, (w, m, v) in enumerate(before):
            w2, ew, m2, em, v2, ev = formula(w, gs[i], m, v, step, **HP)
            got = plan.master[i] if master else ps[i]
            if not master and param == torch.bfloat16:
                ew = ew + 2.0 ** -8 * (w2.abs() + ew)
            assert ((got.double() - w2).abs() <= ew).all(), (i, step)
            assert ((plan.m[i].double() - m2).abs() <= em).all() and ((plan.v[i].double() - v2).abs() <= ev).all()
            if master:
                assert torch.equal(ps[i], plan.master[i].to(torch.bfloat16))


def quantised(codes, scale, value, err, nearest, nonzero):
    """The e4m3 numbers of one tensor against the values (and their error) they stand for."""
    n = value.numel()
    blocks = -(-n // 256)
    pad = lambda x: torch.nn.functional.pad(x, (0, blocks * 256 - n)).view(blocks, 256)  # noqa: E731
    value, err, q = pad(value.cpu()), pad(err.cpu()), pad(codes.cpu().float().double())
    top = value.abs().amax(1)
    assert ((scale.cpu().double() - top / 448).abs() <= err.amax(1) / 448 + 4 * U * top / 448).all()
    x = (value.abs() / scale.cpu().double().clamp(min=1e-300)[:, None]).clamp(max=448)
    slack = (err / scale.cpu().double().clamp(min=1e-300)[:, None]) + x * 8 * U
    x = torch.where(scale.cpu().double()[:, None] > 0, x, torch.zeros_like(x))
    slack = torch.where(scale.cpu().double()[:, None] > 0, slack, torch.zeros_like(x))
    hi = GRID[torch.searchsorted(GRID, (x - slack).clamp(min=0)).clamp(max=126)]
    lo = GRID[(torch.searchsorted(GRID, x + slack, right=True) - 1).clamp(min=0)]
    low, high = torch.minimum(lo, hi), torch.maximum(lo, hi)
    a = q.abs()
    ok = (a == low) | (a == high) | ((a >= low) & (a <= high))
    if nonzero:
        ok &= (a > 0) | (value == 0)
    assert ok.all()
    assert ((q == 0) | (torch.sign(q) == torch.sign(value))).all()
    if nearest:
        step = torch.where(x >= 2.0 ** -6, 2.0 ** (torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3), torch.full_like(x, 2.0 ** -9))
        near = (a - x).abs() <= step / 2 + slack
        if nonzero:
            near |= (a == 2.0 ** -9) & (x < 2.0 ** -9)
        assert near.all()


@pytest.mark.parametrize("seed", [None, 7])
@pytest.mark.parametrize("param,master", [(torch.float32, False), (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("sizes", [[1], [256, 511], [255, 0, 257, 4096, 3, 33333], [5] * 340])
def test_e4m3_moments(sizes, param, master, seed):
    ps = tensors(sizes, param, 2)
    plan = api.adamw_plan(ps, E4M3, master=master)
    for step in (1, 2, 3):
        gs = [g * torch.exp(2 * torch.randn(g.numel(), device="cuda", generator=torch.Generator(device="cuda").manual_seed(step)))
              for g in tensors(sizes, torch.float32, 20 + step, 0.1)]
        before = [((plan.master[i] if master else p).clone(), *moments(plan, i)) for i, p in enumerate(ps)]
        api.adamw_step(plan, gs, step=step, seed=None if seed is None else seed + step, **HP)
        for i, (w, m, v) in enumerate(before):
            w2, ew, m2, em, v2, ev = formula(w, gs[i], m, v, step, **HP)
            # m and sqrt(v) of the step before are products of two floats rounded once more
            em, ev, ew = em + 2 * U * m.abs(), ev + 4 * U * v, ew * 2
            got = plan.master[i] if master else ps[i]
            if not master and param == torch.bfloat16:
                ew = ew + (2.0 ** -7 if seed is not None else 2.0 ** -8) * (w2.abs() + ew)
            assert ((got.double() - w2).abs() <= ew).all(), (i, step)
            if w.numel():
                quantised(plan.m[i], plan.m_scale[i], m2, em, seed is None, False)
                root = v2.sqrt()
                quantised(plan.v[i], plan.v_scale[i], root, ev / (2 * root).clamp(min=1e-30) + U * root, seed is None, True)


def test_random_rounding_keeps_the_expectation():
    """The mean over seeds of m, sqrt(v) and a bf16 weight is the value before
    rounding: within 6 standard deviations of a mean of K numbers that lie a
    step apart (at most step / (2 sqrt(K)) each)."""
    n, K = 512, 400
    g = tensors([n], torch.float32, 3, 0.1)
    w = tensors([n], torch.bfloat16, 4)[0]
    sums = torch.zeros(3, n, dtype=torch.float64, device="cuda")
    for k in range(K):
        p = w.clone()
        plan = api.adamw_plan([p], E4M3)
        api.adamw_step(plan, g, step=1, seed=1000 + k, **HP)
        m, v = moments(plan, 0)
        sums += torch.stack((m, v.sqrt(), p.double()))
    w2, _, m2, _, v2, _ = formula(w, g[0], torch.zeros(n, device="cuda").double(), torch.zeros(n, device="cuda").double(), 1, **HP)
    for got, want, scale, step in ((sums[0] / K, m2, plan.m_scale[0], 2.0 ** -3), (sums[1] / K, v2.sqrt(), plan.v_scale[0], 2.0 ** -3),
                                   (sums[2] / K, w2, None, 2.0 ** -7)):
        least = 0.0 if scale is None else scale.double().repeat_interleave(256) * 2.0 ** -9
        dev = torch.maximum(want.abs() * step, torch.as_tensor(least, device="cuda")) / (2 * math.sqrt(K))
        # sqrt(v) is kept from 0, which lifts what lies under the smallest number to it
        lifted = 0.0 if scale is None else scale.double().repeat_interleave(256) * 2.0 ** -9 * (want.abs() < least)
        assert ((got - want).abs() <= 6 * dev + lifted).all()


def test_moments_move_under_random_rounding():
    """beta2 near 1 changes v by far less than a step of e4m3.  In blocks whose
    largest element holds still (so that the scale does), nearest leaves the
    others where they are, and random rounding follows their decay in the mean
    (each draw errs by at most 2^-4, 16128 elements and 200 steps average)."""
    n = 256 * 64
    first_g = torch.linspace(0.5, 0.9, n, device="cuda")
    first_g[::256] = 1.0
    later = torch.zeros(n, device="cuda")
    later[::256] = 0.001 ** 0.5  # v = 0.001 stays what it is
    rest = torch.arange(n, device="cuda") % 256 != 0
    mean = {}
    for seed in (None, 5):
        p = torch.zeros(n, device="cuda")
        plan = api.adamw_plan([p], E4M3)
        api.adamw_step(plan, [first_g], step=1, lr=0.0, beta2=0.999, seed=seed)
        first = moments(plan, 0)[1].sqrt()[rest].mean()
        for k in range(200):
            api.adamw_step(plan, [later], step=2 + k, lr=0.0, beta2=0.999, seed=None if seed is None else seed + k)
        mean[seed] = (moments(plan, 0)[1].sqrt()[rest].mean() / first).item()
    assert abs(mean[5] - 0.999 ** 100) < 0.02
    assert mean[None] > 0.99


def dither(place, seed):
    """The 32 random bits of each place, from the definition."""
    x = ((place & 0xffffffff) * 0x9e3779b1 + (place >> 32) * 0x85ebca77) & 0xffffffff
    x = x ^ seed
    x = ((x ^ (x >> 16)) * 0x2c1b3c6d) & 0xffffffff
    x = ((x ^ (x >> 12)) * 0x297a2d39) & 0xffffffff
    return x ^ (x >> 15)


@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e7])
def test_e4m3_codes_bit_for_bit(scale):
    """Codes and scales are those of the update in fp32 with one rounding an
    operation, two steps in a row: at ordinary sizes, and for blocks whose
    scales pass what a float holds times 2^120."""
    n, b1, b2 = 256 * 200, 0.9, 0.95
    place = torch.arange(n, device="cuda")
    p = torch.zeros(n, device="cuda")
    plan = api.adamw_plan([p], E4M3)
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")

    def coded(x, rnd, keep):
        x, rnd = x.view(-1, 256), rnd.view(-1, 256)
        top = x.abs().amax(1)
        y = (x.abs() * (448.0 / top)[:, None]).clamp(max=448.0)
        big = ((y.view(torch.int32).long() + (rnd << 4)) >> 20) - 960
        code = torch.where(y >= 2.0 ** -6, big, (y * 512 + rnd.float() / 65536).floor().long())
        if keep:
            code = torch.where((y > 0) & (code == 0), 1, code)
        value = code.to(torch.uint8).view(E4M3).float() * torch.where(x < 0, -1.0, 1.0)
        s = top * (1.0 / 448)
        return value.flatten(), s, (value * s[:, None]).flatten()
    for step in (1, 2):
        g = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(step)) * scale
        api.adamw_step(plan, [g], step=step, seed=step, lr=0.0, beta1=b1, beta2=b2)
        m, v = m * b1 + g * (1 - b1), v * b2 + g * g * (1 - b2)
        bits = dither(place, step)
        cm, sm, m = coded(m, bits & 0xffff, False)
        cv, sv, root = coded(v.sqrt(), bits >> 16, True)
        v = root * root
        assert torch.equal(plan.m_scale[0], sm) and torch.equal(plan.v_scale[0], sv)
        # below 2^-6 the sum with the random bits is rounded elsewhere: a code in a million may differ there
        for got, want in ((plan.m[0].float(), cm), (plan.v[0].float(), cv)):
            assert torch.equal(got[want.abs() >= 2.0 ** -5], want[want.abs() >= 2.0 ** -5])
            assert (got - want).abs().max() <= 2.0 ** -9


def test_one_place_one_random_number():
    """Tensors of a plan draw from one stream: cut at block borders, they get the same bits."""
    n = 256 * 10
    w, g = tensors([n], torch.float32, 5)[0], tensors([n], torch.float32, 6)[0]
    a = [w.clone()]
    pa = api.adamw_plan(a, E4M3)
    b = [w[:768].clone(), w[768:1024].clone(), w[1024:].clone()]
    pb = api.adamw_plan(b, E4M3)
    for step in (1, 2):
        api.adamw_step(pa, [g], step=step, seed=9, **HP)
        api.adamw_step(pb, [g[:768], g[768:1024], g[1024:]], step=step, seed=9, **HP)
    assert torch.equal(a[0], torch.cat(b))
    for x, y in ((pa.m, pb.m), (pa.v, pb.v)):
        assert torch.equal(x[0].view(torch.uint8), torch.cat([t.view(torch.uint8) for t in y]))


@pytest.mark.parametrize("state", [torch.float32, E4M3])
def test_unaligned_tensors_give_the_same_bits(state):
    n = 3000
    w, g = tensors([n], torch.float32, 7)[0], tensors([n], torch.float32, 8)[0]
    out = []
    for off in (0, 1, 3):
        store, gs = torch.zeros(n + 8, device="cuda"), torch.zeros(n + 8, device="cuda")
        p, gg = store[off:off + n], gs[off:off + n]
        p.copy_(w)
        gg.copy_(g)
        plan = api.adamw_plan([p], state)
        api.adamw_step(plan, [gg], step=1, seed=3, **HP)
        assert not store[:off].any() and not store[off + n:].any()
        out.append((p.clone(), plan.m[0].view(torch.uint8).clone(), plan.v[0].view(torch.uint8).clone()))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, out[0]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[], [0], [1], [7, 0, 300, 256], [100003, 5], [3] * 700, [4000003]])
def test_grad_norm(sizes, dtype):
    gs = tensors(sizes, dtype, 11, 0.3)
    want = math.sqrt(sum(float(g.double().square().sum()) for g in gs))
    # squares and a chain of at most (elements of a thread) + 20 fp32 sums of one sign
    bound = (4 + sum(sizes) / (256 * 1216) + 40) * U
    norm, coef = api.grad_norm(gs, max_norm=0.5).tolist()
    assert abs(norm - want) <= bound * want + 1e-30
    assert abs(coef - min(1.0, 0.5 / (want + 1e-6))) <= (bound + 2 * U) * coef
    again = api.grad_norm(gs, max_norm=0.5).tolist()
    assert again == [norm, coef]
    assert api.grad_norm(gs)[1].item() == 1.0


def test_grad_norm_past_32_bit_offsets():
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[(1 << 31) + 5], g[7] = 3.0, 4.0, 12.0
    assert api.grad_norm([g])[0].item() == 13.0


def test_step_past_32_bit_offsets():
    """A tensor of more than 2^32 bytes: its end is updated like a small one's."""
    n, k = (1 << 31) + 512, 512
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-k:] = tensors([k], torch.bfloat16, 40)[0]
    plan = api.adamw_plan([p], E4M3)
    api.adamw_step(plan, [g], step=1, **HP)
    q = torch.zeros(k, dtype=torch.bfloat16, device="cuda")
    small = api.adamw_plan([q], E4M3)
    api.adamw_step(small, [g[-k:].clone()], step=1, **HP)
    assert torch.equal(p[-k:], q) and not p[:1 << 20].any()
    assert torch.equal(plan.m[0].view(torch.uint8)[-k:], small.m[0].view(torch.uint8))


def test_gradient_scale_and_non_finite_gradients():
    p = tensors([1000], torch.float32, 12)
    plan = api.adamw_plan(p)
    g = tensors([1000], torch.float32, 13)
    norm = api.grad_norm(g, max_norm=1.0)
    w = p[0].clone()
    api.adamw_step(plan, g, step=1, grad_scale=norm[1:], **HP)
    z = torch.zeros(1000, device="cuda", dtype=torch.float64)
    w2, ew, *_ = formula(w, g[0], z, z, 1, coef=norm[1].item(), **HP)
    assert ((p[0].double() - w2).abs() <= 2 * ew).all()
    for bad in (float("nan"), float("inf")):
        before = [p[0].clone(), plan.m[0].clone(), plan.v[0].clone()]
        g[0][37] = bad
        norm = api.grad_norm(g, max_norm=1.0)
        assert not torch.isfinite(norm).any()
        api.adamw_step(plan, g, step=2, grad_scale=norm[1:], **HP)
        assert all(torch.equal(a, b) for a, b in zip(before, (p[0], plan.m[0], plan.v[0])))
    api.adamw_step(plan, g, step=2, **HP)  # unscaled, an infinite gradient is the caller's
    assert not torch.isfinite(p[0][37]) and torch.isfinite(p[0][:37]).all()


def test_graph_replays_with_new_scalars():
    w, g = tensors([5000], torch.float32, 14)[0], tensors([5000], torch.float32, 15)[0]
    a, b = w.clone(), w.clone()
    pa, pb = api.adamw_plan([a], E4M3), api.adamw_plan([b], E4M3)
    sc = torch.zeros(4, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        api.adamw_step(pa, [g], step=1, seed=0, scalars=sc, **HP)
    for step in (1, 2, 3):
        sc.copy_(api.adamw_scalars(HP["lr"] / step, step, HP["beta1"], HP["beta2"], HP["weight_decay"], seed=step))
        graph.replay()
        api.adamw_step(pb, [g], step=step, seed=step, **{**HP, "lr": HP["lr"] / step})
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(pa.m[0].view(torch.uint8), pb.m[0].view(torch.uint8))


def test_mixed_types_in_one_plan_and_another_stream():
    ps = [*tensors([300], torch.float32, 16), *tensors([500, 20], torch.bfloat16, 17)]
    gs = [*tensors([300], torch.bfloat16, 18), *tensors([500], torch.float32, 19), *tensors([20], torch.bfloat16, 20)]
    alone = []
    for p, g in zip(ps, gs):
        q = p.clone()
        api.adamw_step(api.adamw_plan([q]), [g], step=1, **HP)
        alone.append(q)
    plan = api.adamw_plan(ps)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.adamw_step(plan, gs, step=1, **HP)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, ps))


def test_checkpointed_moments_continue_bit_for_bit():
    sizes = [700, 256]
    ws = tensors(sizes, torch.bfloat16, 21)
    a = [w.clone() for w in ws]
    pa = api.adamw_plan(a, E4M3)
    for step in (1, 2):
        api.adamw_step(pa, tensors(sizes, torch.bfloat16, 30 + step), step=step, seed=step, **HP)
    kept = [[t.clone() for t in x] for x in (pa.params, pa.m, pa.v, pa.m_scale, pa.v_scale)]
    pb = api.adamw_plan(kept[0], m=kept[1], v=kept[2], m_scale=kept[3], v_scale=kept[4])
    for plan in (pa, pb):
        api.adamw_step(plan, tensors(sizes, torch.bfloat16, 33), step=3, seed=3, **HP)
    assert all(torch.equal(x, y) for x, y in zip(pa.params, pb.params))
