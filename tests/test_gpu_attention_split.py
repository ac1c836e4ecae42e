"""Which form of bd_attention_decode a batch gets, told by its workspace: a head that several CTAs share
leaves its parts there, a head that one warp takes by itself leaves nothing.  Bounds as in test_gpu_attention.py."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import Pool, randn
from test_gpu_attention import check, run
from test_gpu_attention_forms import widened

pytestmark = pytest.mark.gpu


def run_and_tell(pool, q, window=0):
    """out, lse, and whether parts of heads were left in the workspace."""
    ws = torch.zeros(bd.bd_attention_workspace_size(pool.cache(), *q.shape[:2]), dtype=torch.uint8, device="cuda")
    out, lse = run(pool, q, window=window, ws=ws)
    return out, lse, bool(ws.any())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_the_largest_window_is_no_window(kv):
    pool = Pool([3000], 2, 128, 16, kv, seed=1)
    q = randn((1, 8, 128), 9, 2.0).bfloat16()
    plain = run_and_tell(pool, q)
    for window in (2 ** 31 - 1, 2 ** 31 - 20, 2 ** 30):
        out, lse, split = run_and_tell(pool, q, window)
        check(pool, q, out, lse)
        assert split
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
