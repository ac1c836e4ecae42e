"""The generation example's table of positions for callers without a GPU (none needed here)."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300.decode_step import rope_table


@pytest.mark.parametrize("positions,dim,base", [(1, 2, 1e4), (300, 64, 5e5), (77, 128, 1e4)])
def test_table(positions, dim, base):
    """Cosines and sines of 64-bit angles, rounded once: half a step, 2^-24 of the value, and the angles' own rounding, 300 * 2^-52."""
    got = rope_table(positions, dim, base)
    assert got.shape == (positions, dim) and got.dtype == torch.float32
    a = np.outer(np.arange(positions), np.exp(-2 * np.arange(dim // 2) / dim * np.log(base)))
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    assert np.all(np.abs(got.double().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 300 * 2.0 ** -50)
