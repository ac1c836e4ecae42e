"""How exact the softmax weights are that bd_attention_prompt multiplies V by: as single tokens' are, two 16-bit parts each.

Bounds.  Over bf16 and 8 bits a weight's first part is off by 2^-8 of it at most (half a step of bf16), which the second part, a bf16
number again, holds to 2^-8: 2^-16.  Over 4 bits both are fp16 numbers, 2^-11 each: 2^-22, and half a step of fp16's subnormals, 2^-25, of weights
times 2^12, of which the largest is 1 or more: 2^-37 of the largest value for each key.  The rest as in test_gpu_prompt: 2^-14 for fp32 sums,
2^-18 of the largest score, and the output's rounding, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool, attention
from step_ref import f64, randn
from test_gpu_prompt import KINDS, case, rule_of, run

pytestmark = pytest.mark.gpu


def check(pool, q, new, out, rows=None, scale=None, slopes=None, first=None, prefix=None, cap=0.0, window=0):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, q = f64(out), f64(q)
    part = 2.0 ** -22 if pool.kv == "e2m1" else 2.0 ** -16
    at = 0
    for i, n in enumerate(new):
        k, v = pool.values("k", i), pool.values("v", i)
        for r in range(n):
            if rows is not None and r not in rows and r != n - 1:
                continue
            p = pool.lengths[i] - n + r
            ref, _, mag, big = attention(q[at + r], k, v, p, scale, window, cap, None if slopes is None else f64(slopes),
                                         0 if first is None else int(first[at + r]), 0 if prefix is None else int(prefix[i]))
            tol = 2.0 ** -8 * np.abs(ref) + (part + 2.0 ** -14 + 2.0 ** -18 * big[:, None] + 2.0 ** -19 * cap) * mag + 2.0 ** -100
            if pool.kv == "e2m1":
                tol = tol + 2.0 ** -37 * pool.lengths[i] * np.abs(v).max()
            err = np.abs(out[at + r] - ref)
            assert np.all(err <= tol), (i, r, p, float((err / tol).max()))
        at += n


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(32, 8), (1, 1), (12, 1), (150, 1)])
def test_whole_units(kv, dim, q_heads, kv_heads):
    new, past = [1, 17, 150, 3, 40], [5, 0, 130, 300, 88]
    pool, q = case(kv, dim, q_heads, kv_heads, new, past, seed=q_heads + dim, q_std=0.5)
    out, _ = run(pool, q, new)
    check(pool, q, new, out, rows=set(range(0, 150, 7)))
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_several_units_of_a_cta(kv, dim):
    """More units than SMs, of several blocks each: the first scores of one follow the last weights of the one before."""
    new, past = [700, 650, 3, 300], [0, 300, 900, 513]
    pool, q = case(kv, dim, 16, 16, new, past, seed=dim, q_std=0.5)
    out, _ = run(pool, q, new)
    check(pool, q, new, out, rows=set(range(0, 700, 97)) | {255, 256})


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_pieces(kv, dim):
    pool, q = case(kv, dim, 16, 2, [5, 40], [1900, 900], seed=3, q_std=0.5)
    out, _ = run(pool, q, [5, 40])
    check(pool, q, [5, 40], out)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("kw", [dict(cap=2.0), dict(slopes=True), dict(window=100), dict(cap=2.0, slopes=True, window=70, prefix=True, first=True)], ids=str)
def test_rules(kv, kw):
    new, past = [130, 33, 1, 90], [0, 260, 77, 9]
    pool, q = case(kv, 64, 6, 2, new, past, page=16, seed=5, q_std=0.5)
    rule = rule_of(kw, 6, new, past)
    out, _ = run(pool, q, new, **rule)
    check(pool, q, new, out, rows=set(range(0, 130, 9)), **rule)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_as_single_tokens(kv, dim):
    """A prompt's last tokens and the same tokens one at a time differ by no more than the roundings of either's output, 2^-7 of the
    value, and twice what sums and scores are off by (scores are below 8: 2^-14 + 2^-15, and two parts' 2^-16)."""
    lengths = [700, 33, 1, 129]
    pool = Pool(lengths, 2, dim, 16, kv, seed=11)
    q = randn((4, 8, dim), 12, 0.3).bfloat16()
    prompt, lse = run(pool, q, [1] * 4)
    out, lse1 = torch.empty_like(prompt), torch.empty_like(lse)
    cache = pool.cache()
    bd.bd_attention_decode(cache, q.cuda(), torch.from_numpy(pool.table).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), out,
                           torch.zeros(bd.bd_attention_workspace_size(cache, 4, 8), dtype=torch.uint8, device="cuda"), lse=lse1)
    a, b = f64(prompt), f64(out)
    for i, n in enumerate(lengths):
        _, _, mag, big = attention(f64(q[i]), pool.values("k", i), pool.values("v", i), n - 1, dim ** -0.5)
        assert big.max() < 8
        tol = 2.0 ** -7 * np.maximum(np.abs(a[i]), np.abs(b[i])) + 2 * (2.0 ** -14 + 2.0 ** -15 + 2.0 ** -16) * mag
        if kv == "e2m1":
            tol = tol + 2.0 ** -36 * n * np.abs(pool.values("v", i)).max()
        assert np.all(np.abs(a[i] - b[i]) <= tol), i
    assert (lse - lse1).abs().max() <= 2.0 ** -13
