"""Offsets out of order: the sequences that are left out, the rows of the others, and that no two sequences share a row."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from test_gpu_prompt import case, run

pytestmark = pytest.mark.gpu


def taken(offsets, total):
    """(sequence, first row, rows) of those that are attended to."""
    return [(i, a, b - a) for i, (a, b) in enumerate(zip(offsets, offsets[1:])) if 0 <= a <= b <= total and a >= max(offsets[:i + 1])]


@pytest.mark.parametrize("kv", ["bf16", "e2m1"])
@pytest.mark.parametrize("offsets", [[0, 30, 10, 50], [5, 20, 50], [0, 30, 10, 50, 30, 70], [0, 80, 20, 50], [0, -5, 50, 60], [10, 0, 10, 30], [3, 3, 0, 0, 40],
                                     [0, 20, 10, 15, 20, 45]], ids=str)
def test_offsets_out_of_order(kv, offsets):
    n, total = len(offsets) - 1, 70
    pool, q = case(kv, 64, 4, 2, [0] * n, [90 + 7 * i for i in range(n)], page=16, seed=2)
    q = torch.randn((total, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16()
    out, lse = run(pool, q, None, offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    written = torch.zeros(total, dtype=torch.bool)
    for i, first, rows in taken(offsets, total):
        assert not written[first:first + rows].any()
        written[first:first + rows] = True
        new = [rows if j == i else 0 for j in range(n)]
        want, want_lse = run(pool, q[first:first + rows], new)
        assert torch.equal(out[first:first + rows], want) and torch.equal(lse[first:first + rows], want_lse), i
    assert (out[~written] == 3).all() and (lse[~written] == 3).all()
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("at", [3, 31, 32, 40, 98])
def test_disorder_among_many_sequences(at):
    """More than one lot of 32 sequences, their offsets out of order from one of them on: back to a row before it, then as they were."""
    rng = np.random.default_rng(at)
    new, past = rng.integers(1, 4, 100).tolist(), rng.integers(0, 60, 100).tolist()
    pool, q = case("bf16", 64, 2, 1, new, past, page=16, seed=7)
    want, _ = run(pool, q, new)
    offsets = np.concatenate([[0], np.cumsum(new)]).tolist()
    offsets[at] = offsets[max(0, at - 3)]
    out, _ = run(pool, q, None, offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    written = torch.zeros(q.shape[0], dtype=torch.bool)
    for i, first, rows in taken(offsets, q.shape[0]):
        assert rows == new[i]
        written[first:first + rows] = True
    assert torch.equal(out[written], want[written]) and (out[~written] == 3).all()
    assert bd.bd_get_device_status() == bd.BD_OK
