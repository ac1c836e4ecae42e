"""bd_attention_decode over an 8-bit cache whose values' scales differ widely between tokens.

A token with large values has zeros in half of the columns, where the others' small values are all there is: their
weights times their scales are 2^-12 to 2^-24 of the largest and still enter to 2^-16 of themselves.  Bounds as in
test_gpu_attention.py, which hold column by column."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import Pool, randn
from test_gpu_attention import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ratio", [12, 16, 20, 24])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(8, 2), (12, 1)])
@pytest.mark.parametrize("lengths,pages", [([1, 40, 200, 17], None), ([300, 33, 2, 700], 400)])
def test_small_values_beside_large_ones(ratio, dim, q_heads, kv_heads, lengths, pages):
    """In whole heads to a warp, and split over CTAs and joined; weights nearly equal."""
    pool = Pool(lengths, kv_heads, dim, 16, "e4m3", seed=ratio, k_std=0.1)
    pool.v_scale[:] = 127 - ratio
    raw = pool.v.view(torch.uint8)
    for i, n in enumerate(lengths):
        for t in {0, n // 2, n - 1} if n > 3 else {}:
            page, slot = pool.table[i, t // 16], t % 16
            pool.v_scale[page, :, slot] = 127
            raw[page, :, slot, dim // 2:] = 0
    if pages:
        wide = np.full((len(lengths), pages), -1, np.int32)
        wide[:, :pool.table.shape[1]] = pool.table
        pool.table = wide
    q = randn((len(lengths), q_heads, dim), 9).bfloat16()
    out, lse = run(pool, q)
    check(pool, q, out, lse)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("lengths,pages", [([1, 40, 200, 17], None), ([300, 33, 2, 700], 400)])
@pytest.mark.parametrize("byte", [0, 1, 66])
def test_a_cache_of_zeros(byte, lengths, pages):
    """Slots that were never written, values and scale bytes zero (or a byte below the smallest scale's): zeros, and the
    lse of scores that are all zero."""
    pool = Pool(lengths, 2, 64, 16, "e4m3", seed=1)
    for x in (pool.k, pool.v):
        x.view(torch.uint8)[:] = 0
    pool.k_scale[:], pool.v_scale[:] = byte, byte
    if pages:
        wide = np.full((len(lengths), pages), -1, np.int32)
        wide[:, :pool.table.shape[1]] = pool.table
        pool.table = wide
    q = randn((len(lengths), 8, 64), 9).bfloat16()
    out, lse = run(pool, q)
    assert (out == 0).all()
    # log(n): the sum is exact, the logarithm and a product round
    assert np.all(np.abs(lse.cpu().double().numpy() - np.log(lengths)[:, None]) <= 2.0 ** -18)
