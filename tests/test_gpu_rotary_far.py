"""The rotary table at the far end of its declared bound, 2^-22 of the amplitude where position times frequency is below 2^27,
against frequencies and remainders in 50 digits.

To the bound fp32's rounding of the entry is added, 2^-24 of the value."""
import decimal
import math

import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd

pytestmark = pytest.mark.gpu
D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


def rows_of(rows, dim, base, factor=1.0, original=0.0, low=1.0, high=4.0):
    out = np.empty((len(rows), dim))
    with decimal.localcontext(prec=50):
        for i in range(dim // 2):
            f = (D(base).ln() * D(-2 * i) / D(dim)).exp()
            keep = min(max((D(original) * f / (2 * PI) - D(low)) / (D(high) - D(low)), D(0)), D(1))
            f = f * (keep + (1 - keep) / D(factor))
            assert max(rows) * f < 2 ** 27
            for r, p in enumerate(rows):
                turns = p * f / (2 * PI)
                a = float((turns - int(turns)) * 2 * PI)
                out[r, i], out[r, dim // 2 + i] = math.cos(a), math.sin(a)
    return out


@pytest.mark.parametrize("positions,dim,kw", [(1 << 27, 8, dict(base=1e4)), (1 << 26, 12, dict(base=5e5, factor=32.0, original=8192.0)),
                                              (1 << 15, 16, dict(base=1e-4)), (1 << 17, 6, dict(base=1e4, factor=1e-3)), (1 << 24, 20, dict(base=0.5))], ids=str)
def test_far_end(positions, dim, kw):
    t = torch.empty((positions, dim), device="cuda")
    bd.bd_rotary_table(t, **kw)
    rows = sorted({0, 1, 54321 % positions, positions // 3, positions - 1} | set(range(positions - 40, positions)))
    want = rows_of(rows, dim, **kw)
    got = t[torch.tensor(rows, device="cuda")].cpu().double().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -22 + 2.0 ** -24 * np.abs(want))
