"""A page table of no columns: sequences of which nothing is cached yet, whose empty tensor has no address."""
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import Pool, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_nothing_cached_yet(kv):
    cache = Pool([20], 2, 64, 16, kv, seed=1).cache()
    table = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = randn((3, 4, 64), 2).bfloat16().cuda()
    ws = torch.zeros(bd.bd_attention_workspace_size(cache, 3, 4), dtype=torch.uint8, device="cuda")
    for lengths, status in ((i32(0, 0, 0), bd.BD_OK), (i32(0, 5, 0), bd.BD_ERR_BAD_INDEX)):
        out, lse = torch.full_like(q, 3.0), torch.full((3, 4), 3.0, device="cuda")
        bd.bd_attention_decode(cache, q, table, lengths, out, ws, lse=lse)
        assert bd.bd_get_device_status() == status
        assert (out == 0).all() and torch.isneginf(lse).all()
    before = cache.k.clone(), cache.v.clone()
    x = randn((2, 2, 64), 3).bfloat16().cuda()
    for positions, status in ((i32(-1, -1), bd.BD_OK), (i32(-1, 0), bd.BD_ERR_BAD_INDEX)):
        bd.bd_kv_append(cache, None, x, x, positions, table, None, None)
        assert bd.bd_get_device_status() == status
    assert torch.equal(cache.k.view(torch.uint8), before[0].view(torch.uint8)) and torch.equal(cache.v.view(torch.uint8), before[1].view(torch.uint8))
    k, v = (torch.full((2, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    bd.bd_kv_read(cache, table, i32(0, 0, 0, 0), k, v)
    assert bd.bd_get_device_status() == bd.BD_OK and (k == 3).all()
    bd.bd_kv_read(cache, table, i32(0, 1, 1, 2), k, v)
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX and (k == 0).all() and (v == 0).all()
