"""Scores far below their cap: their error is relative to them, not to the cap.

Bounds.  A capped score is within 2^-19 of itself (the series' next term and four roundings where it is below 0.31 of cap, else 2^-21 of cap), and a
score's sum within 2^-19 of scale * sum |q k|, which is no less; so those of test_gpu_prompt_weights and test_gpu_four_bits_weights with twice
the score's part, 2^-17 of the largest score, and nothing of cap.  The statistic: 2^-19 of itself and of the 16 that a logarithm adds, and
2^-18 of the largest score for its error, 2^-18 for the cap's."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool, attention
from step_ref import f64, randn
from test_gpu_four_bits import decode
from test_gpu_prompt import KINDS, run

pytestmark = pytest.mark.gpu


def check(pool, q, positions, seqs, out, lse, cap, scale):
    part = 2.0 ** -22 if pool.kv == "e2m1" else 2.0 ** -16
    for i in range(q.shape[0]):
        n = positions[i] + 1
        k, v = pool.values("k", seqs[i], n), pool.values("v", seqs[i], n)
        ref, ref_lse, mag, big = attention(f64(q[i]), k, v, n - 1, scale, cap=cap)
        tol = 2.0 ** -8 * np.abs(ref) + (part + 2.0 ** -14 + 2.0 ** -17 * big[:, None]) * mag
        if pool.kv == "e2m1":
            tol = tol + 2.0 ** -37 * n * np.abs(v).max()
        assert np.all(np.abs(f64(out[i]) - ref) <= tol), i
        assert np.all(np.abs(f64(lse[i]) - ref_lse) <= 2.0 ** -19 * (np.abs(ref_lse) + 16) + 2.0 ** -17 * big), i


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("cap,q_std", [(1e3, 1.0), (2.0 ** 20, 1.0), (2.0 ** 100, 1.0), (1e3, 40.0), (50.0, 0.01), (2.0 ** -10, 2.0 ** -18)])
def test_scores_below_their_cap(kv, dim, cap, q_std):
    lengths = [150, 300]
    pool = Pool(lengths, 2, dim, 16, kv, seed=4)
    q = randn((70, 8, dim), 5, q_std).bfloat16()
    rule = dict(cap=cap, scale=dim ** -0.5)
    out, lse = run(pool, q, [40, 30], **rule)
    positions, seqs = list(range(110, 150)) + list(range(270, 300)), [0] * 40 + [1] * 30
    check(pool, q, positions, seqs, out.cpu(), lse.cpu(), **rule)
    out, lse = decode(pool, q[[39, 69]], **rule)
    check(pool, q[[39, 69]], [149, 299], [0, 1], out.cpu(), lse.cpu(), **rule)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", KINDS)
def test_scores_on_either_side_of_the_series(kv):
    """One key of one nonzero element: scores of 2^-12 to 2 caps, both signs, in prompts and for single tokens.

    Over 8 and 4 bits weights are taken times 2^15 or 2^12, so that the statistic is (top - 15) + log2(2^15) in base 2: where top is below 1 the
    difference, the logarithm (a step of fp32 below 16) and the sum are off by 2^-21, 2^-20 and 2^-21, together 2^-19 (times log 2)."""
    cap, dim = 32.0, 64
    pool = Pool([1], 1, dim, 16, kv, seed=4)
    k = torch.zeros_like(randn((pool.table.max() + 3, 1, 16, dim), 0))
    k[:, :, :, 0] = 1.0
    pool.set("k", k)
    x = torch.cat([torch.exp2(torch.linspace(-7, 6, 500)), -torch.exp2(torch.linspace(-7, 6, 500))]).bfloat16()
    q = torch.zeros((1, 1000, dim))
    q[0, :, 0] = x.float()
    q = q.bfloat16()
    want = cap * np.tanh(f64(x) * float(pool.values("k", 0)[0, 0, 0]) / cap)
    for _, lse in (run(pool, q, [1], cap=cap, scale=1.0), decode(pool, q, cap=cap, scale=1.0)):
        assert np.all(np.abs(f64(lse)[0] - want) <= 2.0 ** -19 * np.abs(want) + (0 if kv == "bf16" else 2.0 ** -19))
