"""How exact the softmax weights of single tokens are over a 4-bit cache: two fp16 parts, as two 16-bit parts over the other caches.

Bounds.  A part is off by half a step, 2^-11, the two by 2^-22 of the weight, or by half a step of fp16's subnormals, 2^-25, of weights times 2^15, of
which the largest is 2^15 times 1: 2^-40 of it for each key, 2^-39 n times the largest value with the sum in the denominator at least the largest
weight.  The rest as in test_gpu_four_bits: 2^-14 for fp32 sums, 2^-18 of the largest score, 2^-8 of the value for the output's rounding."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool, attention
from step_ref import f64, randn
from test_gpu_four_bits import decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(32, 8), (1, 1), (12, 1), (48, 2)])
@pytest.mark.parametrize("lengths", [[1, 5, 33, 200, 0, 129], [1900, 3, 700]])  # a head to a warp, split over CTAs
@pytest.mark.parametrize("kw", [dict(), dict(cap=2.0, slopes=True)], ids=str)
def test_weights(dim, q_heads, kv_heads, lengths, kw):
    pool = Pool(lengths, kv_heads, dim, 16, "e2m1", seed=q_heads)
    q = randn((len(lengths), q_heads, dim), 9, 0.5).bfloat16()
    cap, slopes = kw.get("cap", 0.0), None
    if kw:
        slopes = torch.full((q_heads,), 0.01)
    out, _ = decode(pool, q, cap=cap, slopes=slopes)
    out = f64(out)
    for i, n in enumerate(lengths):
        v = pool.values("v", i)
        ref, _, mag, big = attention(f64(q[i]), pool.values("k", i), v, n - 1, dim ** -0.5, cap=cap, slopes=None if slopes is None else f64(slopes))
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -22 + 2.0 ** -14 + 2.0 ** -18 * big[:, None] + 2.0 ** -19 * cap) * mag
        tol = tol + 2.0 ** -39 * n * (np.abs(v).max() if n else 0) + 2.0 ** -100
        err = np.abs(out[i] - ref)
        assert np.all(err <= tol), (i, n, float((err / tol).max()))
    assert bd.bd_get_device_status() == bd.BD_OK
