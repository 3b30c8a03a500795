"""AdamW and the gradient norm where they can go wrong beside the update
itself: tensors that move, their types, and magnitudes near the ends of fp32.
Bounds as in test_gpu_adamw.py."""
import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api
from test_gpu_adamw import E4M3, HP, dither, formula, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state", [torch.float32, E4M3])
def test_a_step_follows_tensors_that_moved(state):
    """Weights, master copies and moments whose storage was replaced are updated where they are now, and the old
    storage stays as it was."""
    sizes = [700, 256, 3]
    ws = tensors(sizes, torch.bfloat16, 21)
    a, b = [w.clone() for w in ws], [w.clone() for w in ws]
    pa, pb = (api.adamw_plan(x, state, master=True) for x in (a, b))
    for step in (1, 2, 3):
        for ts in (b, pb.master, pb.m, pb.v, *((pb.m_scale, pb.v_scale) if state == E4M3 else ())):
            old = ts[1].data
            ts[1].data = ts[1].detach().clone()
            old.view(torch.uint8).fill_(7)
        gs = tensors(sizes, torch.bfloat16, 30 + step)
        for plan in (pa, pb):
            api.adamw_step(plan, gs, step=step, seed=step, **HP)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert all(torch.equal(x, y) for x, y in zip(pa.master, pb.master))
        for x, y in ((pa.m, pb.m), (pa.v, pb.v)):
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(x, y))


@pytest.mark.parametrize("state", [torch.float32, E4M3])
def test_master_copies_of_the_bf16_weights_of_a_mixed_model(state):
    """bf16 matrices and fp32 norms in one plan: master=True keeps copies of the former alone, and every tensor is
    updated as in a plan of its own."""
    sizes, types = [300, 5000, 20, 1], [torch.float32, torch.bfloat16, torch.float32, torch.bfloat16]
    ps = [tensors([n], t, 16 + i)[0] for i, (n, t) in enumerate(zip(sizes, types))]
    gs = tensors(sizes, torch.float32, 18)
    alone = []
    for p, g in zip(ps, gs):
        q = p.clone()
        one = api.adamw_plan([q], state, master=p.dtype == torch.bfloat16)
        api.adamw_step(one, [g], step=1, **HP)
        alone.append((q, one.master))
    plan = api.adamw_plan(ps, state, master=True)
    assert [x is None for x in plan.master] == [True, False, True, False]
    api.adamw_step(plan, gs, step=1, **HP)
    for p, copy, (q, other) in zip(ps, plan.master, alone):
        assert torch.equal(p, q) and (copy is None or torch.equal(copy, other[0]))
    again = api.adamw_plan(ps, m=plan.m, v=plan.v, m_scale=plan.m_scale, v_scale=plan.v_scale, master=plan.master)
    api.adamw_step(again, gs, step=2, **HP)


def coded(x, rnd, keep):
    """x as e4m3 numbers, scales and the values they stand for, in fp32 with one rounding an operation."""
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


def check_codes(magnitude, zeros=False):
    """Two steps' codes and scales against the same update in torch fp32: equal from 2^-5 on, at most one number apart
    below (there the sum with the random bits is rounded elsewhere)."""
    n, b1, b2 = 256 * 200, 0.9, 0.95
    plan = api.adamw_plan([torch.zeros(n, device="cuda")], E4M3)
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for step in (1, 2):
        g = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(step)) * magnitude
        if zeros:
            g[::3] = 0
        api.adamw_step(plan, [g], step=step, seed=step, lr=0.0, beta1=b1, beta2=b2)
        m, v = m * b1 + g * (1 - b1), v * b2 + g * g * (1 - b2)
        bits = dither(torch.arange(n, device="cuda"), step)
        cm, sm, m = coded(m, bits & 0xffff, False)
        cv, sv, root = coded(v.sqrt(), bits >> 16, True)
        v = root * root
        assert torch.equal(plan.m_scale[0], sm) and torch.equal(plan.v_scale[0], sv)
        for got, want in ((plan.m[0].float(), cm), (plan.v[0].float(), cv)):
            assert torch.equal(got[want.abs() >= 2.0 ** -5], want[want.abs() >= 2.0 ** -5])
            assert (got - want).abs().max() <= 2.0 ** -9


@pytest.mark.parametrize("magnitude,zeros", [(1e-14, False), (1e-16, False), (1e-17, True), (1e-18, False), (3e-19, True)])
def test_square_roots_of_small_second_moments(magnitude, zeros):
    """v from 1e-28 down to subnormal numbers, and zeros beside them: the stored roots are those of sqrt in fp32."""
    check_codes(magnitude, zeros)


@pytest.mark.parametrize("magnitude,zeros", [(1e5, False), (1e14, True), (1e17, False), (1e18, True), (3e18, False)])
def test_moments_of_large_gradients(magnitude, zeros):
    """Scales from 64 up to the largest root of a finite v, and zero codes beside them."""
    check_codes(magnitude, zeros)


def test_first_moments_up_to_the_end_of_fp32():
    """Without gradients v stays 0, and m is halved wherever it lies in fp32."""
    n = 256 * 8
    x = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    for top in (1e20, 1e30, 3.3e38):
        m, ms, kept = coded(x / x.abs().max() * top, torch.full((n,), 0x8000, device="cuda"), False)
        plan = api.adamw_plan([torch.zeros(n, device="cuda")], m=[m.to(E4M3)], v=[torch.zeros(n, device="cuda").to(E4M3)],
                              m_scale=[ms], v_scale=[torch.zeros(n // 256, device="cuda")])
        api.adamw_step(plan, [torch.zeros(n, device="cuda")], step=1, lr=0.0, beta1=0.5)
        want, s, _ = coded(kept * 0.5, torch.full((n,), 0x8000, device="cuda"), False)
        assert torch.equal(plan.m_scale[0], s)
        big = want.abs() >= 2.0 ** -5
        assert torch.equal(plan.m[0].float()[big], want[big]) and (plan.m[0].float() - want).abs().max() <= 2.0 ** -9


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("magnitude", [1e-40, 1e-25, 1e-15, 1e15, 1e25, 1e36])
@pytest.mark.parametrize("sizes", [[1], [3, 5000, 300], [100003, 0, 256]])
def test_norms_whose_squares_leave_fp32(sizes, magnitude, dtype):
    """Squares above 2^128 and below 2^-149, beside zeros and values of ordinary size: the norm of a float is a float.
    Bound as in test_grad_norm; a subnormal norm is held to 2^-149."""
    gs = [torch.randn(n, generator=torch.Generator().manual_seed(n)).double().mul_(magnitude).to(dtype).cuda() for n in sizes]
    gs.append(torch.zeros(70000, dtype=dtype, device="cuda"))
    for extra in ([], [torch.ones(2000, dtype=dtype, device="cuda")]):
        both = [g for pair in zip(extra, gs) for g in pair] + gs[len(extra):]
        want = sum(float(g.double().square().sum()) for g in both) ** 0.5
        norm, coef = api.grad_norm(both, max_norm=0.5).tolist()
        bound = (4 + (sum(sizes) + 72000) / (256 * 1216) + 40) * 2.0 ** -24
        assert abs(norm - want) <= bound * want + 2.0 ** -149
        assert abs(coef - min(1.0, 0.5 / (want + 1e-6))) <= (bound + 2.0 ** -23) * coef
        assert api.grad_norm(both, max_norm=0.5).tolist() == [norm, coef]


def test_norms_that_are_not_finite():
    g = torch.ones(70000, device="cuda")
    for bad in (float("inf"), float("nan"), -float("inf")):
        g[12345] = bad
        assert not torch.isfinite(api.grad_norm([g], max_norm=1.0)).any()
    g.fill_(3e38)  # finite gradients, but a norm that fp32 does not hold
    norm, coef = api.grad_norm([g], max_norm=1.0).tolist()
    assert norm == float("inf") and coef != coef


def test_a_step_with_large_gradients_is_clipped():
    """A gradient of 1e25 scales to the norm that was asked for and the step is taken."""
    p = torch.zeros(1000, device="cuda")
    g = torch.full((1000,), 1e25, device="cuda")
    norm = api.grad_norm([g], max_norm=1.0)
    plan = api.adamw_plan([p])
    api.adamw_step(plan, [g], lr=1.0, step=1, grad_scale=norm[1:])
    assert torch.allclose(p, torch.full_like(p, -1.0), rtol=1e-5)  # m / sqrt(v) of equal gradients


def test_autograd_sees_that_a_step_changed_the_weights():
    """A backward pass through weights that were updated since the forward pass is refused, as for any in-place change."""
    w = torch.nn.Parameter(torch.ones(300, device="cuda"))
    plan = api.adamw_plan([w])
    loss = (w * w).sum()
    api.adamw_step(plan, [torch.ones(300, device="cuda")], lr=0.1, step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    (w * w).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach())
    with torch.inference_mode():
        p = torch.ones(300, device="cuda")
        api.adamw_step(api.adamw_plan([p]), [torch.ones(300, device="cuda")], lr=0.1, step=1)
    assert torch.equal(p, w.detach())


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [255, 0, 257, 5000]])
def test_random_rounding_of_bf16_weights_with_fp32_moments(sizes, grad):
    """bf16 weights without a master copy go up or down to a neighbour of the updated weight, by the bits of their
    places, and keep its expectation: the mean of K draws lies within 6 standard deviations, a step / (2 sqrt(K)) each."""
    K = 200
    ws = tensors(sizes, torch.bfloat16, 50)
    gs = tensors(sizes, grad, 51, 0.1)
    zero = [torch.zeros(n, device="cuda", dtype=torch.float64) for n in sizes]
    sums = [z.clone() for z in zero]
    for k in range(K):
        ps = [w.clone() for w in ws]
        plan = api.adamw_plan(ps)
        api.adamw_step(plan, gs, step=1, seed=100 + k, **HP)
        for i, (p, w, g) in enumerate(zip(ps, ws, gs)):
            w2, ew, *_ = formula(w, g, zero[i], zero[i], 1, **HP)
            assert ((p.double() - w2).abs() <= ew + 2.0 ** -7 * (w2.abs() + ew)).all()
            sums[i] += p.double()
    for i, (w, g) in enumerate(zip(ws, gs)):
        w2, ew, *_ = formula(w, g, zero[i], zero[i], 1, **HP)
        assert ((sums[i] / K - w2).abs() <= ew + 6 * 2.0 ** -7 * (w2.abs() + ew) / (2 * K ** 0.5)).all()
    ps, qs = [w.clone() for w in ws], [w.clone() for w in ws]
    for x in (ps, qs):
        api.adamw_step(api.adamw_plan(x), gs, step=1, seed=9, **HP)
    assert all(torch.equal(a, b) for a, b in zip(ps, qs))


def test_gradients_from_a_generator():
    ws, gs = tensors([300, 20], torch.float32, 60), tensors([300, 20], torch.float32, 61)
    assert torch.equal(api.grad_norm((g for g in gs), max_norm=1.0), api.grad_norm(gs, max_norm=1.0))
    a, b = [w.clone() for w in ws], [w.clone() for w in ws]
    api.adamw_step(api.adamw_plan(a), gs, step=1, **HP)
    api.adamw_step(api.adamw_plan(w for w in b), (g for g in gs), step=1, **HP)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
