"""bd_kv_append and bd_kv_read on the GPU.

The write is defined down to its roundings, so the cache's bytes are compared with a CPU form
in fp32 exactly; against 64 bits a rotated value is off by at most 3 roundings of its two products and
the one to the stored type.  Reading back is exact."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import Pool, f64, quantised, randn, rotated, rotated_f32

pytestmark = pytest.mark.gpu


def rope_table(n, dim):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(dim // 2) / (dim // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def bits(t):
    return t.contiguous().cpu().view(torch.uint8 if t.element_size() == 1 else torch.int16)


def expected(pool, k, v, seq, pos):
    """The pool after the write: k and v fp32 rows on the CPU."""
    out = {n: (None if getattr(pool, n) is None else getattr(pool, n).clone()) for n in ("k", "v", "k_scale", "v_scale")}
    for i, (s, p) in enumerate(zip(seq, pos)):
        if p < 0:
            continue
        page, slot = int(pool.table[s, p // pool.page]), p % pool.page
        for n, x in (("k", k[i]), ("v", v[i])):
            if pool.kv == "bf16":
                out[n][page, :, slot] = x.bfloat16()
            else:
                val, byte = quantised(x)
                out[n].view(torch.uint8)[page, :, slot] = val.view(torch.uint8)
                out[n + "_scale"][page, :, slot] = byte
    return out


def append(pool, q, k, v, seq, pos, rope, in_place=False):
    cache = pool.cache()
    qd = None if q is None else q.cuda()
    qo = None if q is None else (qd if in_place else torch.full_like(qd, 9.0))
    bd.bd_kv_append(cache, qd, k.cuda(), v.cuda(), torch.tensor(pos, dtype=torch.int32).cuda(),
                    torch.from_numpy(pool.table).cuda(), None if rope is None else rope.cuda(), qo,
                    seq_ids=None if seq is None else torch.tensor(seq, dtype=torch.int32).cuda())
    return cache, qo


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,q_heads,kv_heads,page", [(128, 32, 8, 16), (128, 5, 5, 48), (64, 12, 4, 16), (64, 7, 1, 1024),
                                                       (128, 64, 8, 64), (64, 1, 1, 32)])
def test_append_writes_the_defined_bytes(kv, dim, q_heads, kv_heads, page):
    lengths = [1, page, page + 1, 3 * page - 1, 40]
    pool = Pool(lengths, kv_heads, dim, page, kv, seed=dim + page)
    # a whole prompt, one token, the last slot of a page and the first of the next
    seq = [4] * 40 + [0, 1, 2, 2, 3]
    pos = list(range(40)) + [0, page - 1, page, 0, 2 * page]
    t = len(seq)
    q, k, v = (randn((t, h, dim), 5 + h, s).bfloat16() for h, s in ((q_heads, 1.0), (kv_heads, 3.0), (kv_heads, 0.01)))
    k[3, 0] = 0  # a row of zeros
    v[4, 0, 0] = 2.0 ** 100  # the rest of its row goes to zero
    rope = rope_table(max(pos) + 1, dim)
    cache, qo = append(pool, q, k, v, seq, pos, rope)
    turned = rope[torch.tensor(pos)]
    assert torch.equal(bits(qo), bits(rotated_f32(q, turned).bfloat16()))
    ref = rotated(f64(q), f64(turned))
    size = rotated(np.abs(f64(q)), np.abs(f64(turned)))  # not |ac| + |bs| in its first half
    size[..., : dim // 2] = (np.abs(f64(q))[..., : dim // 2] * np.abs(f64(turned))[:, None, : dim // 2]
                             + np.abs(f64(q))[..., dim // 2:] * np.abs(f64(turned))[:, None, dim // 2:])
    assert np.all(np.abs(f64(qo) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size)
    want = expected(pool, rotated_f32(k, turned), v.float(), seq, pos)
    for n, w in want.items():
        if w is not None:
            assert torch.equal(bits(getattr(cache, n)), bits(w)), n
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_without_rotation_and_without_seq_ids(kv):
    pool = Pool([5, 17, 33], 2, 64, 16, kv, seed=1)
    k, v = randn((3, 2, 64), 2).bfloat16(), randn((3, 2, 64), 3).bfloat16()
    cache, _ = append(pool, None, k, v, None, [4, 16, 32], None)
    want = expected(pool, k.float(), v.float(), [0, 1, 2], [4, 16, 32])
    for n, w in want.items():
        if w is not None:
            assert torch.equal(bits(getattr(cache, n)), bits(w)), n


def test_append_in_place_query_and_padding():
    pool = Pool([5, 17, 33], 2, 128, 16, "e4m3", seed=1)
    q, k, v = (randn((3, h, 128), 4 + h).bfloat16() for h in (6, 2, 2))
    rope = rope_table(64, 128)
    cache, qo = append(pool, q, k, v, [0, 1, 2], [4, -1, 32], rope, in_place=True)
    want_q = rotated_f32(q, rope[[4, 0, 32]]).bfloat16()
    want_q[1] = q[1]  # a skipped token's row stays
    assert torch.equal(bits(qo), bits(want_q))
    want = expected(pool, rotated_f32(k, rope[[4, 0, 32]]), v.float(), [0, 1, 2], [4, -1, 32])
    for n, w in want.items():
        assert torch.equal(bits(getattr(cache, n)), bits(w)), n
    assert bd.bd_get_device_status() == bd.BD_OK


def test_scale_edges():
    """Powers of two, 448 times them, one bf16 step beyond, zero, the smallest and largest values, infinity, NaN."""
    inf, nan = float("inf"), float("nan")
    tops = [448.0, 450.0, 1.0, 1.75, 1.7578125, 0.0, 2.0 ** -133, 2.0 ** -60, 1.5 * 2.0 ** -52, 2.0 ** 127, 3.3e38, inf, nan, -3.5]
    pool = Pool([len(tops)], 1, 64, 16, "e4m3", seed=0)
    k = randn((len(tops), 1, 64), 7, 1e-3).bfloat16()
    for i, t in enumerate(tops):
        k[i] *= 0 if t == 0 else 1
        if 0 < abs(t) < 1e-10:
            k[i] = 0
        k[i, 0, 5] = t
    pos = list(range(len(tops)))
    cache, _ = append(pool, None, k, k, [0] * len(tops), pos, None)
    want = expected(pool, k.float(), k.float(), [0] * len(tops), pos)
    for n in ("k_scale", "v_scale"):
        assert torch.equal(getattr(cache, n).cpu(), want[n])
    for n in ("k", "v"):
        got, ref = getattr(cache, n).cpu().float(), want[n].float()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))


@pytest.mark.parametrize("what", ["page", "page_high", "seq", "position", "rope"])
def test_append_bad_index_flags_and_skips(what):
    pool = Pool([40, 40], 2, 64, 16, "bf16", seed=1)
    if what == "page":
        pool.table[1, 0] = -1
    if what == "page_high":
        pool.table[1, 0] = pool.k.shape[0]
    seq = [0, 2 if what == "seq" else 1]
    pos = [3, {"position": 48, "rope": 40}.get(what, 5)]
    k = randn((2, 2, 64), 2).bfloat16()
    q = randn((2, 4, 64), 2).bfloat16()
    rope = rope_table(40, 64)
    cache, qo = append(pool, q, k, k, seq, pos, rope)
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    want = expected(pool, rotated_f32(k, rope[[3, 0]]), k.float(), [0, 1], [3, -1])
    assert torch.equal(bits(cache.k), bits(want["k"])) and torch.equal(bits(cache.v), bits(want["v"]))
    assert (qo[1] == 9).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,kv_heads,page", [(128, 8, 16), (64, 3, 32), (128, 1, 48), (64, 32, 1024)])
def test_read_is_exact(kv, dim, kv_heads, page):
    lengths = [0, 1, page, 0, page + 1, 5, 100, 0]
    pool = Pool(lengths, kv_heads, dim, page, kv, seed=3, junk=0x7F if kv == "e4m3" else float("nan"))
    total = sum(lengths)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    out = [torch.full((total + 3, kv_heads, dim), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    bd.bd_kv_read(pool.cache(), torch.from_numpy(pool.table).cuda(), off, *out)
    for n, got in zip("kv", out):
        ref = np.concatenate([pool.values(n, i) for i in range(len(lengths))])
        assert np.array_equal(f64(got[:total]), ref)
        assert (got[total:] == 5).all()
    assert bd.bd_get_device_status() == bd.BD_OK


def test_read_bad_page_gives_zeros_and_flags():
    pool = Pool([20, 20], 2, 64, 16, "e4m3", seed=3)
    pool.table[0, 1] = -7
    off = torch.tensor([0, 20, 60], dtype=torch.int32).cuda()  # the second sequence asks beyond its table
    out = [torch.empty((60, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    bd.bd_kv_read(pool.cache(), torch.from_numpy(pool.table).cuda(), off, *out)
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    k = f64(out[0])
    assert np.array_equal(k[:16], pool.values("k", 0, 16)) and not k[16:20].any()
    assert np.array_equal(k[20:40], pool.values("k", 1)) and not k[52:].any()


def test_pools_beyond_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^32: written, read and attended to at the far end."""
    heads, page, dim = 8, 64, 128
    n_pages = (1 << 32) // (heads * page * dim) + 16  # over 2^32 elements, 8.6 GB a pool
    k, v = (torch.empty((n_pages, heads, page, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    cache = bd.KVCache(k, v)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32).cuda()
    n = 3 * page - 5
    kn, vn, q = randn((n, heads, dim), 1).bfloat16(), randn((n, heads, dim), 2).bfloat16(), randn((1, 16, dim), 3).bfloat16()
    bd.bd_kv_append(cache, None, kn.cuda(), vn.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), table, None, None,
                    seq_ids=torch.zeros(n, dtype=torch.int32, device="cuda"))
    ko, vo = (torch.empty((n, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    bd.bd_kv_read(cache, table, torch.tensor([0, n], dtype=torch.int32).cuda(), ko, vo)
    assert torch.equal(ko.cpu(), kn) and torch.equal(vo.cpu(), vn)
    from step_ref import attention
    out = torch.empty((1, 16, dim), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(bd.bd_attention_workspace_size(cache, 1, 16), dtype=torch.uint8, device="cuda")
    bd.bd_attention_decode(cache, q.cuda(), table, torch.tensor([n], dtype=torch.int32).cuda(), out, ws)
    ref, _, mag, big = attention(f64(q[0]), f64(kn), f64(vn), dim ** -0.5)
    assert np.all(np.abs(f64(out[0]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -14 + 2.0 ** -18 * big[:, None]) * mag)
    assert bd.bd_get_device_status() == bd.BD_OK


def test_refusals():
    pool = Pool([5], 2, 64, 16, "e4m3", seed=1)
    d = pool.device()
    for bad in (dict(k_scale=None), dict(v=d["v"][:1]), dict(k=d["k"].float()), dict(k_scale=d["k_scale"].int())):
        with pytest.raises(ValueError):
            bd.KVCache(**{**d, **bad})
    with pytest.raises(ValueError):
        bd.KVCache(torch.empty((2, 2, 16, 64), dtype=torch.bfloat16, device="cuda"),
                   torch.empty((2, 2, 16, 64), dtype=torch.bfloat16, device="cuda"), d["k_scale"], d["v_scale"])
    cache = pool.cache()
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.from_numpy(pool.table).cuda()
    for args in ((None, k[:, :1], k, pos, table, None, None), (None, k, k, pos.long(), table, None, None),
                 (None, k, k, pos, table[0], None, None), (None, k, k.float(), pos, table, None, None),
                 (None, k, k, pos, table, torch.zeros((4, 32), device="cuda"), None)):
        with pytest.raises(ValueError):
            bd.bd_kv_append(cache, *args)
    with pytest.raises(bd.BitDeltaError) as e:  # a query needs a rotation
        bd.bd_kv_append(cache, k, k, k, pos, table, None, k)
    assert e.value.status == bd.BD_ERR_INVALID_ARG
    for page, dim, status in ((8, 64, bd.BD_ERR_UNSUPPORTED_SHAPE), (16, 96, bd.BD_ERR_UNSUPPORTED_SHAPE),
                              (2048, 64, bd.BD_ERR_UNSUPPORTED_SHAPE)):
        x = torch.zeros((1, 1, page, dim), dtype=torch.bfloat16, device="cuda")
        y = torch.zeros((1, 1, dim), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(bd.BitDeltaError) as e:
            bd.bd_kv_append(bd.KVCache(x, x.clone()), None, y, y, pos, table, None, None)
        assert e.value.status == status
