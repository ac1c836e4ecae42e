"""bd_attention_decode where every key is streamed by CTAs and joined, and where each warp takes whole heads.

Which of the two runs follows from what the page table's width and the window allow a sequence to
hold, so the same short lengths are run under a narrow table and under a wide one.  Bounds as in test_gpu_attention.py."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import Pool, randn
from test_gpu_attention import check, run

pytestmark = pytest.mark.gpu


def widened(pool, pages):
    """The same pool under a table of `pages` columns; the new ones hold no valid id."""
    wide = np.full((pool.table.shape[0], pages), -1, np.int32)
    wide[:, :pool.table.shape[1]] = pool.table
    pool.table = wide
    return pool


@pytest.mark.parametrize("pages", [3, 400])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(32, 8), (4, 4), (16, 1), (48, 2), (9, 3)])
def test_short_sequences(pages, kv, dim, q_heads, kv_heads):
    lengths = [1, 0, 15, 16, 17, 31, 32, 33, 0, 64, 65, 96] * 3
    pool = widened(Pool(lengths, kv_heads, dim, 32, kv, seed=dim + q_heads, junk=0x7F if kv == "e4m3" else float("nan")), pages)
    q = randn((len(lengths), q_heads, dim), 9, 2.0).bfloat16()
    out, lse = run(pool, q)
    check(pool, q, out, lse)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_more_heads_than_warps(kv):
    """300 sequences of 8 KV heads: some warps take a second head."""
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 49, 300).tolist()
    pool = Pool(lengths, 8, 128, 16, kv, seed=4)
    q = randn((300, 32, 128), 9, 2.0).bfloat16()
    out, lse = run(pool, q)
    check(pool, q, out, lse, seqs=list(range(0, 300, 13)) + [298, 299])
    again, lse2 = run(pool, q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 17, 40])
def test_many_windows(kv, window):
    """A window keeps long sequences short; pages before it have no valid id."""
    lengths = [200, 0, 5, 333, 40, 41, 16, 1, 100, 64] * 6
    pool = Pool(lengths, 8, 128, 16, kv, seed=window)
    for i, n in enumerate(lengths):
        pool.table[i, :max(0, n - window) // 16] = -7
    table, pool.table = pool.table, np.maximum(pool.table, 0)
    values = {(x, i): pool.values(x, i) for x in ("k", "v") for i in range(len(lengths))}
    pool.values = lambda x, i, n=None: values[x, i]
    pool.table = table
    q = randn((len(lengths), 16, 128), 9, 2.0).bfloat16()
    out, lse = run(pool, q, window=window)
    check(pool, q, out, lse, window=window)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("pages", [4, 400])
def test_bad_page_and_length(pages):
    """A page id out of range drops its keys, a negative length the sequence; both are reported."""
    lengths = [40, 64, 10] * 8
    pool = widened(Pool(lengths, 4, 128, 16, "bf16", seed=8), pages)
    good = pool.table.copy()
    pool.table[1, 2] = 10 ** 6
    q = randn((len(lengths), 8, 128), 9, 2.0).bfloat16()
    given = list(lengths)
    given[2] = -3
    out, lse = run(pool, q, lengths=given)
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    pool.table = good
    check(pool, q, out, lse, seqs=[0] + list(range(3, 24)))
    kept = Pool.values

    class Cut:
        lengths = pool.lengths

        @staticmethod
        def values(name, i, n=None):
            x = kept(pool, name, i, n)
            return np.concatenate([x[:32], x[48:]])
    check(Cut, q, out, lse, seqs=[1])
