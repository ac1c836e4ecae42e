"""bd_rmsnorm with the sum written over x or over the residual: the bits of a call with buffers of its own."""
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from test_gpu_step_norm import EPS, cuda, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [8, 256, 512, 1000, 2048, 4096, 8192, 14336, 32768])
@pytest.mark.parametrize("over", ["x", "residual", "x without a residual"])
def test_sum_in_place(n, over):
    x, r, w, ids = (cuda(v) for v in make(33, n, 3, over != "x without a residual", seed=n))
    y, y2, sum2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    bd.bd_rmsnorm(x, w, EPS, y2, residual=r, residual_out=sum2, weight_ids=ids)
    target = r if over == "residual" else x
    for _ in range(2 if r is None else 1):  # without a residual the sum is x, again and again
        bd.bd_rmsnorm(x, w, EPS, y, residual=r, residual_out=target, weight_ids=ids)
        assert torch.equal(y, y2) and torch.equal(target, sum2)
    assert bd.bd_get_device_status() == bd.BD_OK
