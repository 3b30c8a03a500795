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
