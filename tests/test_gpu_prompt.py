"""bd_attention_prompt on the GPU against the definition in 64 bits.

Bounds.  A score is added up by the tensor cores in steps whose sums may be truncated: within 2^-19 of scale * sum |q k| (and
2^-21 of cap; distances enter with a relative 2^-22), so a weight is within twice that (numerator and sum).  Weights are rounded to bf16, 2^-8 of each, and
accumulated in fp32, 2^-14 with exp2 and the scale: (2^-8 + 2^-14 + 2^-18 * max_j |score| + 2^-19 * cap) * sum p |v|.  The
output's rounding to bf16 is 2^-8 of the value.  Weights below fp32's normal range, 2^-126 of at least 2^-8 of the largest, become 0: fewer than
2^14 of them, of values below 2^4, are off by less than 2^-100.  Over a 4-bit cache weights are fp16 numbers times 2^12: half a step of its
subnormals is 2^-25, so that each is off by up to 2^-37 of the largest weight beside its 2^-11: 2^-37 n max|v| more."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool, attention
from step_ref import f64, randn

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "e2m1"]


def offsets_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()


def run(pool, q, new, lengths=None, offsets=None, table=None, ws=None, stream=None, **rule):
    cache = pool.cache() if isinstance(pool, Pool) else pool
    lengths = pool.lengths if lengths is None else lengths
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    if ws is None:
        ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, q.shape[1]), dtype=torch.uint8, device="cuda")
    rule = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in rule.items()}
    bd.bd_attention_prompt(cache, q.cuda(), offsets_of(new) if offsets is None else offsets,
                           torch.from_numpy(pool.table).cuda() if table is None else table,
                           torch.tensor(lengths, dtype=torch.int32).cuda(), out, ws, lse=lse, stream=stream, **rule)
    return out, lse


def check(pool, q, new, out, lse, rows=None, scale=None, slopes=None, first=None, prefix=None, cap=0.0, window=0):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse, q = f64(out), f64(lse), f64(q)
    at = 0
    for i, n in enumerate(new):
        k, v = pool.values("k", i), pool.values("v", i)
        for r in range(n):
            if rows is not None and r not in rows and r != n - 1:
                continue
            p = pool.lengths[i] - n + r
            ref, ref_lse, mag, big = attention(q[at + r], k, v, p, scale, window, cap, None if slopes is None else f64(slopes),
                                               0 if first is None else int(first[at + r]), 0 if prefix is None else int(prefix[i]))
            err = np.abs(out[at + r] - ref)
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -18 * big[:, None] + 2.0 ** -19 * cap) * mag + 2.0 ** -100
            if pool.kv == "e2m1" and pool.lengths[i]:
                tol = tol + 2.0 ** -37 * pool.lengths[i] * np.nanmax(np.abs(v))
            assert np.all(err <= tol), (i, r, p, float((err - tol).max()), float(err.max()))
            if np.isneginf(ref_lse).any():
                assert (out[at + r] == 0).all() and np.isneginf(lse[at + r]).all(), (i, r, p)
            else:
                assert np.all(np.abs(lse[at + r] - ref_lse) <= 2.0 ** -19 * (np.abs(ref_lse) + 16 + cap) + 2.0 ** -18 * big), (i, r, p)
        at += n


def case(kv, dim, q_heads, kv_heads, new, past, page=32, seed=0, q_std=2.0, **kw):
    pool = Pool([a + b for a, b in zip(new, past)], kv_heads, dim, page, kv, seed, **kw)
    return pool, randn((sum(new), q_heads, dim), seed + 9, q_std).bfloat16()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(32, 8), (4, 4), (8, 1), (1, 1), (12, 1), (48, 2), (9, 3), (150, 1)])
def test_heads_and_lengths(kv, dim, q_heads, kv_heads):
    """One token to several tiles, nothing new, nothing cached before; slots that no token uses hold NaN."""
    new, past = [1, 0, 17, 70, 3, 0, 40], [0, 5, 0, 130, 300, 0, 88]
    pool, q = case(kv, dim, q_heads, kv_heads, new, past, seed=q_heads + dim, junk=True)
    out, lse = run(pool, q, new)
    check(pool, q, new, out, lse)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("page", [16, 48, 64, 1024])
def test_pages_and_long_prompts(kv, page):
    new, past = [900, 1, 513], [0, 700, 300]
    pool, q = case(kv, 128, 8, 2, new, past, page=page, seed=page, junk=True)
    out, lse = run(pool, q, new)
    check(pool, q, new, out, lse, rows=set(range(0, 900, 61)) | {63, 64, 127, 128})


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("new,past", [([5], [9000]), ([40, 1], [3000, 5000]), ([1, 1, 2], [2100, 0, 700])])
def test_few_queries_over_many_keys(kv, new, past):
    """Keys are split over CTAs and joined; the same bits each time, with a workspace used before."""
    pool, q = case(kv, 128, 16, 2, new, past, seed=3)
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(pool.cache(), 16), dtype=torch.uint8, device="cuda")
    first = run(pool, q, new, ws=ws)
    check(pool, q, new, *first)
    small, sq = case(kv, 128, 16, 2, [3], [20], seed=4)
    check(small, sq, [3], *run(small, sq, [3], ws=ws))
    again = run(pool, q, new, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


RULES = [dict(cap=20.0), dict(slopes=True), dict(window=1), dict(window=100), dict(window=5000), dict(prefix=True), dict(first=True),
         dict(cap=5.0, slopes=True, window=70, prefix=True, first=True), dict(scale=-0.3), dict(scale=0.0), dict(scale=2.0),
         dict(first=True, prefix=True, window=33)]


def rule_of(kw, heads, new, past, seed=0):
    rng = np.random.default_rng(seed)
    rule = dict(kw)
    if kw.get("slopes"):
        rule["slopes"] = torch.from_numpy(rng.normal(0.1, 0.2, heads).astype(np.float32))
    if kw.get("prefix"):
        rule["prefix"] = torch.tensor([[-3, 1 << 30, (a + b) // 2][i % 3] for i, (a, b) in enumerate(zip(new, past))], dtype=torch.int32)
    if kw.get("first"):
        f = np.concatenate([rng.integers(-5, n + p + 2, n) for n, p in zip(new, past)])
        f[::7] = 1 << 30
        rule["first"] = torch.from_numpy(f.astype(np.int32))
    return rule


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("kw", RULES, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_rules(kv, kw):
    new, past = [130, 0, 33, 1, 90], [0, 40, 260, 77, 9]
    pool, q = case(kv, 64, 6, 2, new, past, page=16, seed=5, junk=True)
    rule = rule_of(kw, 6, new, past)
    out, lse = run(pool, q, new, **rule)
    check(pool, q, new, out, lse, **rule)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
def test_unseen_infinities_and_nan(kv, dim):
    """A token whose K and V are NaN reaches only the queries that see it; keys before the window have no page."""
    new, past = [200, 90], [0, 300]
    pool, q = case(kv, dim, 4, 2, new, past, page=16, seed=6, junk=True)
    pool.spoil_tokens(0, [150]), pool.spoil_tokens(1, [200, 201])
    if kv == "bf16":
        t = pool.table[0, 170 // 16]
        pool.v[t, :, 170 % 16, 5] = float("-inf")
    out, lse = run(pool, q, new, window=60)
    clean0 = [r for r in range(200) if r < 150]
    clean1 = [r for r in range(90) if 300 + r - 60 >= 201]
    check_rows = {0: clean0, 1: clean1}
    o, l, qq = f64(out), f64(lse), f64(q)
    at = 0
    for i, n in enumerate(new):
        k, v = pool.values("k", i), pool.values("v", i)
        for r in check_rows[i]:
            p = pool.lengths[i] - n + r
            ref, ref_lse, mag, big = attention(qq[at + r], k, v, p, dim ** -0.5, 60)
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -18 * big[:, None]) * mag
            assert np.all(np.abs(o[at + r] - ref) <= tol), (i, r)
            assert np.all(np.abs(l[at + r] - ref_lse) <= 2.0 ** -19 * (np.abs(ref_lse) + 16) + 2.0 ** -18 * big)
        at += n
    assert np.isnan(o[150:200]).all()
