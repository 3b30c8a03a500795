"""The table of an AdamW plan follows its tensors: what a step hands to the
library, without launching one (the plan's own rows work on any device)."""
import pytest
import torch

from backward_tcgen05_tma_gemms_gb300 import api
from test_abi_host import lib  # noqa: F401  (fixture)


def plan_of(n=5, size=300, state=torch.float32, master=False):
    params = [torch.zeros(size + i, dtype=torch.bfloat16 if master else torch.float32) for i in range(n)]
    moments = [[torch.zeros(p.numel(), dtype=torch.uint8).view(state) if state.itemsize == 1 else torch.zeros(p.numel())
                for p in params] for _ in range(2)]
    scales = [[torch.zeros(-(-p.numel() // 256)) for p in params] if state.itemsize == 1 else None for _ in range(2)]
    return api.AdamWPlan(params, [p.float() for p in params] if master else None, *moments, *scales)


def lists(plan):
    return {"param": plan.params, "master": plan.master, "m": plan.m, "v": plan.v, "m_scale": plan.m_scale,
            "v_scale": plan.v_scale}


@pytest.mark.parametrize("how", ["data", "set_", "entry"])
@pytest.mark.parametrize("state,master", [(torch.float32, False), (torch.float32, True), (torch.float8_e4m3fn, True)])
def test_rows_name_the_storage_that_is_there(how, state, master):
    plan = plan_of(state=state, master=master)
    assert [int(x) for x in plan.rows()["param"]] == [p.data_ptr() for p in plan.params]
    for name, ts in lists(plan).items():
        if ts is None:
            continue
        new = ts[2].detach().clone()
        if how == "data":
            ts[2].data = new
        elif how == "set_":
            ts[2].set_(new)
        else:
            ts[2] = new
        rows = plan.rows()
        for field, now in lists(plan).items():
            assert [int(x) for x in rows[field]] == ([t.data_ptr() for t in now] if now else [0] * 5), (name, field)


def test_old_storage_is_not_handed_out_while_the_table_names_it():
    """A freed storage's address may go to the next tensor of its size; the plan keeps it until it looks again."""
    plan = plan_of(n=1, size=1 << 20)
    plan.rows()
    old = plan.params[0].data_ptr()
    plan.params[0].data = torch.zeros(1 << 20)
    assert torch.zeros(1 << 20).data_ptr() != old
    assert int(plan.rows()["param"][0]) == plan.params[0].data_ptr() != old


def test_moved_tensors_are_checked_again():
    def moved(name, new, **kw):
        plan = plan_of(**kw)
        plan.rows()
        lists(plan)[name][1].data = new
        return plan
    with pytest.raises(TypeError):
        moved("param", torch.zeros(301, dtype=torch.float64)).rows()
    with pytest.raises(ValueError, match="shape"):
        moved("param", torch.zeros(300)).rows()
    with pytest.raises(ValueError, match="shape"):
        moved("m", torch.zeros(302)).rows()
    with pytest.raises(TypeError):
        moved("v", torch.zeros(301, dtype=torch.bfloat16)).rows()
    with pytest.raises(api.TpsError) as e:
        moved("param", torch.zeros(301, 2)[:, 0]).rows()
    assert e.value.code == api.ERR_LAYOUT
    with pytest.raises(ValueError, match="shape"):
        moved("m_scale", torch.zeros(1), state=torch.float8_e4m3fn).rows()


def test_released_storage_is_refused(lib):  # noqa: F811
    """A storage that was resized away has no address: the library refuses the row before any launch."""
    import ctypes
    plan = plan_of(n=1)
    plan.rows()
    plan.params[0].untyped_storage().resize_(0)
    rows = plan.rows()
    rows["grad"] = 0x1000
    h = api.TpsAdamwHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1, 0, 0)
    assert lib.tps_adamw_step(rows.ctypes.data, 1, ctypes.byref(h), None, None, None) == api.ERR_ARG


def test_master_copies_are_for_bf16_weights_alone():
    params = [torch.zeros(300), torch.zeros(500, dtype=torch.bfloat16), torch.zeros(20, dtype=torch.bfloat16)]
    moments = [[torch.zeros(p.numel()) for p in params] for _ in range(2)]
    copies = [None, params[1].float(), None]
    plan = api.AdamWPlan(params, copies, *moments, None, None)
    assert [int(x) for x in plan.rows()["master"]] == [0, copies[1].data_ptr(), 0]
    plan.master[1], plan.master[2] = None, params[2].float()
    assert [int(x) for x in plan.rows()["master"]] == [0, 0, plan.master[2].data_ptr()]
    with pytest.raises(TypeError, match="master"):
        api.AdamWPlan(params, [params[0].clone(), None, None], *moments, None, None).rows()
    with pytest.raises(ValueError, match="shape"):
        api.AdamWPlan(params, [None, params[1].float()], *moments, None, None).rows()
    plan.params.append(torch.zeros(3))
    with pytest.raises(ValueError, match="shape"):
        plan.rows()


def test_a_workspace_the_kernels_cannot_write_is_refused(monkeypatch):
    """One on the host, and one whose elements share storage, never reach the library."""
    with pytest.raises(ValueError, match="GPU"):
        api._room(torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(TypeError):
        api._room(bytearray(16))

    def library():
        raise AssertionError("reached the library")
    monkeypatch.setattr(api, "library", library)
    with pytest.raises(ValueError, match="GPU"):
        api._linear_ce_call(lambda ws, n: library(), 1, 8, 8, torch.float32, False,
                            torch.empty(1 << 20, dtype=torch.uint8), None)


def test_a_tensor_given_twice_is_refused():
    """Two warps would update the same elements at once (a weight that two layers share belongs in the list once)."""
    w, flat = torch.zeros(300), torch.zeros(600)
    moments = lambda n: [torch.zeros(n), torch.zeros(n)]  # noqa: E731
    for params, m, v in (([w, w], moments(300), moments(300)), ([w.clone(), w], [flat[:300], flat[299:599]], moments(300)),
                         ([flat[:300], flat[300:]], moments(300), [flat[:300], torch.zeros(300)])):
        with pytest.raises(ValueError, match="twice"):
            api.AdamWPlan(params, None, m, v, None, None).rows()
    api.AdamWPlan([flat[:300], flat[300:]], None, moments(300), moments(300), None, None).rows()
    plan = plan_of(n=2, size=300)
    plan.rows()
    plan.params[1].data = plan.params[0].data
    with pytest.raises(ValueError):
        plan.rows()
    api.AdamWPlan([torch.zeros(0), torch.zeros(0)], None, [torch.zeros(0)] * 2, [torch.zeros(0)] * 2, None, None).rows()


def test_gradients_that_come_one_by_one(monkeypatch):
    """A generator was walked several times: after the first walk there were no gradients, and their norm was 0."""
    with pytest.raises(ValueError, match="GPU"):
        api.grad_norm(g for g in [torch.zeros(3)])
    g = [torch.zeros(3), torch.zeros(4)]
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    again, ptrs, numels, _, _ = api._grad_list(x for x in g)
    assert list(numels) == [3, 4] and list(ptrs) == [x.data_ptr() for x in g] and again[1] is g[1]
