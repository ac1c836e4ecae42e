"""The 4-bit cache: bytes as defined, read back exactly, and attention of single tokens over it and with a score rule.

Attention's bounds are test_gpu_attention's, except that a 4-bit cache's weights enter as one fp16 number each, 2^-11
(below 2^-29 of the head's largest weight half a step of fp16's subnormals, 2^-40 of it, for each key: 2^-39 n times the largest value with
the sum in the denominator at least the largest weight)."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool, attention, four_bits, four_values
from step_ref import f64, randn

pytestmark = pytest.mark.gpu


def append(pool_shape, x, y=None, page=16):
    """Tokens x (and y for V), [t, heads, dim], one per sequence, at position 3 of a page of its own."""
    t, heads, dim = x.shape
    cache = bd.KVCache(*[torch.full((t, heads, page, w), 7, dtype=torch.uint8, device="cuda") for w in (dim // 2, dim // 2, dim // 16, dim // 16)])
    bd.bd_kv_append(cache, None, x.cuda(), (x if y is None else y).cuda(), torch.full((t,), 3, dtype=torch.int32, device="cuda"),
                    torch.arange(t, dtype=torch.int32, device="cuda")[:, None], None, None)
    return cache


@pytest.mark.parametrize("dim", [64, 128])
def test_bytes_of_every_size(dim):
    """Magnitudes over the whole of bf16's range; ties between codes and between scales; zeros, infinities and NaN."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((400, 3, dim), generator=g) * torch.exp2(torch.randint(-40, 40, (400, 3, 1), generator=g).float())
    x[:100] = torch.randint(-24, 25, (100, 3, dim), generator=g).float() / 4  # many ties
    x[100, :, :16] = 0
    x[101, 0, 3], x[101, 1, 20], x[101, 2, 0] = float("inf"), float("-inf"), float("nan")
    x[102] = 3e38
    x[103] = 1e-38
    x[104, :, :] = 2.0 ** -19
    x = x.bfloat16()
    cache = append(None, x)
    raw, scale = four_bits(x.float())
    for name in "kv":
        pool, s = getattr(cache, name).cpu(), getattr(cache, name + "_scale").cpu()
        assert torch.equal(s[:, :, 3], scale)
        fine = scale != 255
        assert torch.equal(pool[:, :, 3].view(400, 3, -1, 8)[fine], raw.view(400, 3, -1, 8)[fine])
        assert (pool[:, :, [0, 1, 2, 4]] == 7).all() and (s[:, :, [0, 1, 2, 4]] == 7).all()


@pytest.mark.parametrize("dim,heads,page", [(64, 3, 32), (128, 1, 48), (64, 32, 1024), (128, 8, 16)])
def test_read_is_exact(dim, heads, page):
    lengths = [5, 0, 100, 1, 33]
    pool = Pool(lengths, heads, dim, page, "e2m1", seed=dim)
    pool.k_scale.copy_(torch.from_numpy(np.random.default_rng(2).integers(0, 248, pool.k_scale.shape).astype(np.uint8)))
    pool.spoil_tokens(2, [7])
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    out = [torch.full((sum(lengths) + 2, heads, dim), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    bd.bd_kv_read(pool.cache(), torch.from_numpy(pool.table).cuda(), off, *out)
    for name, o in zip("kv", out):
        want = np.concatenate([pool.values(name, i) for i in range(5)])
        assert np.array_equal(f64(o)[:-2], want, equal_nan=True)
        assert (o[-2:] == 5).all()
    assert bd.bd_get_device_status() == bd.BD_OK


def decode(pool, q, lengths=None, ws=None, **rule):
    cache = pool.cache()
    n, heads, _ = q.shape
    out, lse = torch.full_like(q, 3.0, device="cuda"), torch.full((n, heads), 3.0, device="cuda")
    if ws is None:
        ws = torch.zeros(bd.bd_attention_workspace_size(cache, n, heads), dtype=torch.uint8, device="cuda")
    rule = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in rule.items()}
    bd.bd_attention_decode(cache, q.cuda(), torch.from_numpy(pool.table).cuda(),
                           torch.tensor(pool.lengths if lengths is None else lengths, dtype=torch.int32).cuda(), out, ws, lse=lse, **rule)
    return out, lse


def check(pool, q, out, lse, scale=None, slopes=None, first=None, cap=0.0, window=0):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    one = 2.0 ** -11 if pool.kv == "e2m1" else 0.0
    out, lse, q = f64(out), f64(lse), f64(q)
    for i, n in enumerate(pool.lengths):
        ref, ref_lse, mag, big = attention(q[i], pool.values("k", i), pool.values("v", i), n - 1, scale, window, cap,
                                           None if slopes is None else f64(slopes), 0 if first is None else int(first[i]))
        top = np.abs(pool.values("v", i)).max() if n and one else 0.0
        tol = 2.0 ** -8 * np.abs(ref) + (one + 2.0 ** -14 + 2.0 ** -18 * big[:, None] + 2.0 ** -19 * cap) * mag + 2.0 ** -39 * n * top + 2.0 ** -100
        assert np.all(np.abs(out[i] - ref) <= tol), (i, n, float((np.abs(out[i] - ref) - tol).max()))
        if np.isneginf(ref_lse).any():
            assert (out[i] == 0).all() and np.isneginf(lse[i]).all(), i
        else:
            assert np.all(np.abs(lse[i] - ref_lse) <= 2.0 ** -19 * (np.abs(ref_lse) + 16 + cap) + 2.0 ** -18 * big), (i, n)


HEADS = [(32, 8), (4, 4), (8, 1), (1, 1), (12, 1), (16, 1), (48, 2), (9, 3)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", HEADS)
def test_heads_and_lengths(dim, q_heads, kv_heads):
    pool = Pool([1, 0, 15, 16, 17, 63, 64, 65, 0, 200, 129, 2], kv_heads, dim, 32, "e2m1", seed=q_heads, junk=True)
    q = randn((12, q_heads, dim), 9, 2.0).bfloat16()
    check(pool, q, *decode(pool, q))
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("lengths", [[4099, 1, 1000, 0, 2500], [70, 500, 0, 3, 512, 128]])
@pytest.mark.parametrize("kw", [dict(cap=20.0), dict(slopes=True), dict(first=True), dict(cap=5.0, slopes=True, first=True, window=100),
                                dict(slopes=True, scale=-0.2)], ids=str)
@pytest.mark.parametrize("dim,heads", [(64, (6, 2)), (128, (32, 2))])
def test_rules(kv, lengths, kw, dim, heads):
    """Split over CTAs and, where the table is narrow, a head to a warp."""
    pool = Pool(lengths, heads[1], dim, 16, kv, seed=8, junk=True)
    q = randn((len(lengths), heads[0], dim), 9, 2.0).bfloat16()
    rule = dict(kw)
    if kw.get("slopes"):
        rule["slopes"] = torch.from_numpy(np.random.default_rng(1).normal(0.05, 0.1, heads[0]).astype(np.float32))
    if kw.get("first"):
        rule["first"] = torch.tensor([[n // 3, -4, n, 1 << 30, n - 1][i % 5] for i, n in enumerate(lengths)], dtype=torch.int32)
    check(pool, q, *decode(pool, q, **rule), **rule)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("page", [16, 48, 1024])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_pages_windows_and_repeats(page, window):
    pool = Pool([4099, 1, 1000, 0, 2500], 2, 128, page, "e2m1", seed=page, junk=True)
    q = randn((5, 8, 128), 9, 2.0).bfloat16()
    first = decode(pool, q, window=window)
    check(pool, q, *first, window=window)
    again = decode(pool, q, window=window)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_sizes_far_apart():
    """Scales that differ by 2^30 between tokens and groups; queries far from 1; values that nearly vanish beside others."""
    pool = Pool([300, 300, 300], 2, 64, 16, "e2m1", seed=6)
    rng = np.random.default_rng(0)
    pool.k_scale.copy_(torch.from_numpy(rng.integers(60, 130, pool.k_scale.shape).astype(np.uint8)))
    pool.v_scale.copy_(torch.from_numpy(rng.integers(1, 247, pool.v_scale.shape).astype(np.uint8)))
    q = randn((3, 8, 64), 9, 1.0)
    q[1] *= 1e-20
    q[2] *= 30.0
    q = q.bfloat16()
    check(pool, q, *decode(pool, q))


def test_nan_reaches_only_who_sees_it():
    pool = Pool([100, 100], 1, 64, 16, "e2m1", seed=6)
    pool.spoil_tokens(0, [20])
    q = randn((2, 4, 64), 9, 2.0).bfloat16()
    out, _ = decode(pool, q, window=70)
    clean = f64(out)
    ref = attention(f64(q[0]), pool.values("k", 0), pool.values("v", 0), 99, 0.125, 70)[0]
    assert np.abs(clean[0] - ref).max() <= 0.02 * np.abs(ref).max()
    out, _ = decode(pool, q)
    assert torch.isnan(out[0]).all() and not torch.isnan(out[1]).any()


def test_bad_pages_and_lengths_flag():
    pool = Pool([64, 64, 64], 2, 64, 16, "e2m1", seed=2)
    want = decode(pool, randn((3, 4, 64), 9).bfloat16())[0]
    pool.table[1, 2] = 10000
    out, _ = decode(pool, randn((3, 4, 64), 9).bfloat16(), lengths=[64, 64, 100])
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    assert torch.equal(out[0], want[0]) and torch.isfinite(out).all()


def test_four_values_cover_every_code():
    assert np.array_equal(four_values(np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]], np.uint8), np.array([[120]], np.uint8))[0],
                          [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
