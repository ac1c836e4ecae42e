"""The example's unscaled positions on the GPU and its host function give one table: 2^-22 for the first, half a step of fp32 for either."""
import pytest
import torch

from bit_delta_tenant_gb300.decode_step import Shape, Tenants, rope_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("base,dim", [(1e4, 64), (5e5, 128)])
def test_one_table(base, dim):
    shape = Shape(layers=1, hidden=128, q_heads=2, kv_heads=2, head_dim=dim, mlp=128, vocab=100, rope_base=base)
    t = Tenants(shape, 1, [0], 500, page_size=16)
    assert (t.rope.cpu() - rope_table(500, dim, base)).abs().max() <= 2.0 ** -22 + 2.0 ** -23
