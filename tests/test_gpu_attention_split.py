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


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("seqs,kv_heads,longest", [(200, 8, 3001), (57, 32, 777), (224, 8, 6000)])
def test_a_long_sequence_among_short_ones_is_split(kv, seqs, kv_heads, longest):
    """So many heads that they come to one per warp, under a table of 8192 tokens."""
    lengths = np.random.default_rng(seqs).integers(0, 20, seqs).tolist()
    lengths[seqs // 3] = longest
    pool = widened(Pool(lengths, kv_heads, 64, 32, kv, seed=2), 256)
    q = randn((seqs, kv_heads, 64), 9, 2.0).bfloat16()
    out, lse, split = run_and_tell(pool, q)
    assert split
    check(pool, q, out, lse, seqs=[0, 1, seqs // 3, seqs - 1])
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,pages", [(0, 8), (100, 256)])
def test_short_heads_are_taken_whole(kv, window, pages):
    """Under a narrow table, or a wide one with a window; with as many heads as warps."""
    lengths = np.random.default_rng(5).integers(0, 250, 200).tolist()
    pool = widened(Pool(lengths, 8, 64, 32, kv, seed=3), pages)
    q = randn((200, 8, 64), 9, 2.0).bfloat16()
    out, lse, split = run_and_tell(pool, q, window)
    assert not split
    check(pool, q, out, lse, window=window, seqs=[0, 1, 77, 199])
