"""Tokens that are not finite, in blocks that some rows see and others do not: who sees one is NaN, everyone else as if it were not there.

Blocks whose V is not finite are added up row by row.  Cases: tokens that leave a window, of other documents, behind a prefix; in a unit's first block and
in later ones; over pieces; beside keys whose page id is out of range; V alone, so that the statistic stays as it is.  The bounds are
test_gpu_prompt_weights's: two 16-bit parts of a weight, 2^-14 for fp32 sums, 2^-18 of the largest score, the output's rounding."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import f64
from test_gpu_prompt import KINDS, case, run

pytestmark = pytest.mark.gpu


def spoil(pool, i, tokens, values_only):
    if not values_only:
        return pool.spoil_tokens(i, tokens)
    for t in tokens:
        at = (pool.table[i, t // pool.page], slice(None), t % pool.page)
        if pool.kv == "bf16":
            pool.v[at] = float("nan")
        elif pool.kv == "e4m3":
            pool.v.view(torch.uint8)[at] = 0x7F
        else:
            pool.v_scale[at] = 255


def seen_by(p, n, window=0, first=0, prefix=0):
    j = np.arange(n)
    seen = ((j <= p) | (j < prefix)) & (j >= first)
    return seen & (j > p - window) if window else seen


def check(pool, q, new, bad, values_only, out, lse, gone=(), **rule):
    """`bad`: spoiled tokens of each sequence; `gone`: tokens of sequence 0 without a page."""
    dim, out, lse, q = q.shape[2], f64(out), f64(lse), f64(q)
    at, nan_rows = 0, 0
    for i, n in enumerate(new):
        length = pool.lengths[i]
        k, v = pool.values("k", i), pool.values("v", i)
        for r in range(n):
            row = at + r
            seen = seen_by(length - n + r, length, rule.get("window", 0), int(rule["first"][row]) if "first" in rule else 0,
                           int(rule["prefix"][i]) if "prefix" in rule else 0)
            if i == 0:
                seen[list(gone)] = False
            spoiled = seen[bad[i]].any()
            nan_rows += spoiled
            if spoiled and not values_only:
                assert np.isnan(out[row]).all() and np.isnan(lse[row]).all(), (i, r)
                continue
            if not seen.any():
                assert (out[row] == 0).all() and np.isneginf(lse[row]).all(), (i, r)
                continue
            kv_heads = k.shape[1]
            qh = q[row].reshape(kv_heads, -1, dim)
            s = np.einsum("hgd,nhd->hgn", qh, k[seen]) * dim ** -0.5
            big = (np.einsum("hgd,nhd->hgn", np.abs(qh), np.abs(k[seen])) * dim ** -0.5).max(-1).reshape(-1)
            top = s.max(-1, keepdims=True)
            w = np.exp(s - top)
            ref_lse = (top[..., 0] + np.log(w.sum(-1))).reshape(-1)
            assert np.all(np.abs(lse[row] - ref_lse) <= 2.0 ** -19 * (np.abs(ref_lse) + 16) + 2.0 ** -18 * big), (i, r)
            if spoiled:
                assert np.isnan(out[row]).all(), (i, r)
                continue
            w /= w.sum(-1, keepdims=True)
            ref = np.einsum("hgn,nhd->hgd", w, v[seen]).reshape(-1, dim)
            mag = np.einsum("hgn,nhd->hgd", w, np.abs(v[seen])).reshape(-1, dim)
            part = 2.0 ** -22 if pool.kv == "e2m1" else 2.0 ** -16
            tol = 2.0 ** -8 * np.abs(ref) + (part + 2.0 ** -14 + 2.0 ** -18 * big[:, None]) * mag
            if pool.kv == "e2m1":
                tol = tol + 2.0 ** -37 * seen.sum() * np.abs(v[seen]).max()
            assert np.all(np.abs(out[row] - ref) <= tol), (i, r)
        at += n
    assert nan_rows > 0
    return at - nan_rows


def both(test):
    for mark in (pytest.mark.parametrize("kv", KINDS), pytest.mark.parametrize("dim", [64, 128]), pytest.mark.parametrize("values_only", [False, True])):
        test = mark(test)
    return test


@both
def test_a_window_that_has_passed(kv, dim, values_only):
    """Rows 300 .. 389 see 60 keys each: token 250 lies in the first block of all, 270 and 333 in later ones; keys wholly before the window have no page."""
    new, past, bad = [90, 90], [300, 300], [[250, 270], [333]]
    pool, q = case(kv, dim, 4, 2, new, past, page=16, seed=6, q_std=0.5, junk=True)
    for i, tokens in enumerate(bad):
        spoil(pool, i, tokens, values_only)
    table = pool.table.copy()
    table[:, :240 // 16] = [-1, pool.k.shape[0]] * 7 + [-1]
    out, lse = run(pool, q, new, table=torch.from_numpy(table).cuda(), window=60)
    assert bd.bd_get_device_status() == bd.BD_OK
    assert 0 < check(pool, q, new, bad, values_only, out, lse, window=60) < sum(new)


@both
def test_other_documents(kv, dim, values_only):
    """Documents of 37 tokens, one of them spoiled; tokens between documents see nothing."""
    new, past, bad = [200, 50], [0, 130], [[40, 41, 73], [150]]
    pool, q = case(kv, dim, 6, 3, new, past, page=32, seed=7, q_std=0.5, junk=True)
    for i, tokens in enumerate(bad):
        spoil(pool, i, tokens, values_only)
    p = np.concatenate([np.arange(200), np.arange(130, 180)])
    first = torch.from_numpy(np.where(p % 37 == 36, 1 << 30, p // 37 * 37).astype(np.int32))
    out, lse = run(pool, q, new, first=first)
    assert 0 < check(pool, q, new, bad, values_only, out, lse, first=first) < sum(new)
    assert bd.bd_get_device_status() == bd.BD_OK


@both
def test_behind_a_prefix(kv, dim, values_only):
    """Sequence 0's prefix holds none of the spoiled tokens, sequence 1's holds one: every row sees it."""
    new, past, bad = [200, 20], [0, 0], [[120, 160], [15]]
    pool, q = case(kv, dim, 4, 4, new, past, page=16, seed=8, q_std=0.5, junk=True)
    for i, tokens in enumerate(bad):
        spoil(pool, i, tokens, values_only)
    prefix = torch.tensor([100, 18], dtype=torch.int32)
    out, lse = run(pool, q, new, prefix=prefix)
    assert 0 < check(pool, q, new, bad, values_only, out, lse, prefix=prefix) < sum(new)
    assert bd.bd_get_device_status() == bd.BD_OK


@both
def test_beside_keys_without_a_page(kv, dim, values_only):
    """In the block of the spoiled token a page id is out of range; its keys count as unseen."""
    new, past, bad = [90], [100], [[140]]
    pool, q = case(kv, dim, 4, 2, new, past, page=16, seed=9, q_std=0.5, junk=True)
    spoil(pool, 0, bad[0], values_only)
    table = pool.table.copy()
    table[0, 128 // 16], table[0, 176 // 16] = -5, pool.k.shape[0]
    gone = list(range(128, 144)) + list(range(176, 190))
    out, lse = run(pool, q, new, table=torch.from_numpy(table).cuda())
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    bad = [[140, 150]]  # 140 has gone with its page
    spoil(pool, 0, [150], values_only)
    out, lse = run(pool, q, new, table=torch.from_numpy(table).cuda())
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    assert 0 < check(pool, q, new, bad, values_only, out, lse, gone=gone) < sum(new)


@both
@pytest.mark.parametrize("bad,clean", [([[1005, 1020, 2520]], 0), ([[1005, 2530]], 25)])
def test_over_pieces(kv, dim, values_only, bad, clean):
    """Few queries over keys that are split: the first piece's first block and the last piece's last one are seen in part."""
    new, past = [40], [2500]
    pool, q = case(kv, dim, 16, 2, new, past, page=64, seed=10, q_std=0.5, junk=True)
    spoil(pool, 0, bad[0], values_only)
    out, lse = run(pool, q, new, window=1500)
    assert check(pool, q, new, bad, values_only, out, lse, window=1500) == clean
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_values_of_one_column(dim, value):
    """Rows that do not see it are as they were; those that do are not finite in that column and as they were in the others."""
    new = [150]
    pool, q = case("bf16", dim, 4, 2, new, [0], page=16, seed=11, q_std=0.5)
    want, want_lse = run(pool, q, new)
    at = (pool.table[0, 70 // 16], slice(None), 70 % 16, 5)
    pool.v[at] = value
    out, lse = run(pool, q, new)
    assert torch.equal(lse, want_lse)
    assert not torch.isfinite(out[70:, :, 5]).any()
    # the block is added up another way: sums of up to 150 products in another order, 2^-14 of sum p |v|, and a rounding either side of a tie, 2^-7
    v = np.abs(pool.values("v", 0))
    v[70, :, 5] = 0
    gap = np.abs(f64(out) - f64(want))
    gap[70:, :, 5] = 0
    assert np.all(gap <= 2.0 ** -7 * np.abs(f64(want)) + 2.0 ** -13 * v.max())
