"""The decode-step entry points refuse bad arguments before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from bit_delta_tenant_gb300 import bitdelta as bd
from bit_delta_tenant_gb300 import build as bd_build

A = 0x10000   # fake device addresses: never dereferenced on these paths
ODD = A + 8


@pytest.fixture(scope="module")
def lib():
    bd_build.build()
    return bd.load_library()


def test_status_string(lib):
    assert "position" in bd.bd_status_string(bd.BD_ERR_BAD_INDEX)


def test_rmsnorm(lib):
    def call(x=A, r=A, w=A, ids=A, nw=2, m=4, n=256, eps=1e-5, y=A, yt=0, ys=0, sc=0, ro=A):
        return lib.bd_rmsnorm(x, r, w, ids, nw, m, n, eps, y, yt, ys, sc, ro, None)
    for kw in (dict(x=0), dict(w=0), dict(y=0), dict(m=-1), dict(n=0), dict(nw=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(yt=2), dict(ys=A), dict(yt=1, sc=128)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    for kw in (dict(n=12), dict(n=bd.BD_NORM_MAX_N + 8), dict(m=1 << 31), dict(yt=1, ys=A, sc=64),
               dict(yt=1, ys=A, sc=128, n=264)):
        assert call(**kw) == bd.BD_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=ODD), dict(r=ODD), dict(w=ODD), dict(y=ODD), dict(ro=ODD), dict(ids=A + 2), dict(yt=1, ys=A + 1, sc=128)):
        assert call(**kw) == bd.BD_ERR_MISALIGNED, kw
    assert call(m=0, x=0, y=0) == bd.BD_OK


def cache(**kw):
    d = dict(k=A, v=A, k_scale=0, v_scale=0, n_pages=4, kv_heads=2, head_dim=64, page_size=16, kv_type=0)
    d.update(kw)
    c = bd.KVCacheDesc()
    for n, v in d.items():
        setattr(c, n, v)
    return c


BAD_CACHES = [(None, bd.BD_ERR_INVALID_ARG)] + [(cache(**kw), s) for kw, s in (
    (dict(k=0), bd.BD_ERR_INVALID_ARG), (dict(kv_type=2), bd.BD_ERR_INVALID_ARG), (dict(k_scale=A), bd.BD_ERR_INVALID_ARG),
    (dict(kv_type=1), bd.BD_ERR_INVALID_ARG), (dict(kv_type=1, k_scale=A), bd.BD_ERR_INVALID_ARG),
    (dict(n_pages=0), bd.BD_ERR_INVALID_ARG), (dict(kv_heads=0), bd.BD_ERR_INVALID_ARG),
    (dict(head_dim=96), bd.BD_ERR_UNSUPPORTED_SHAPE), (dict(page_size=24), bd.BD_ERR_UNSUPPORTED_SHAPE),
    (dict(page_size=2048), bd.BD_ERR_UNSUPPORTED_SHAPE), (dict(kv_heads=bd.BD_KV_MAX_HEADS + 1), bd.BD_ERR_UNSUPPORTED_SHAPE),
    (dict(v=ODD), bd.BD_ERR_MISALIGNED), (dict(kv_type=1, k_scale=ODD, v_scale=A), bd.BD_ERR_MISALIGNED))]


def test_kv_append(lib):
    def call(c=cache(), q=A, qh=4, k=A, v=A, t=3, seq=A, pos=A, table=A, ns=2, mp=4, rope=A, rl=64, qo=A):
        return lib.bd_kv_append(None if c is None else ctypes.byref(c), q, qh, k, v, t, seq, pos, table, ns, mp, rope, rl, qo, None)
    for c, status in BAD_CACHES:
        assert call(c=c) == status
    for kw in (dict(k=0), dict(v=0), dict(pos=0), dict(table=0), dict(t=-1), dict(ns=-1), dict(mp=-1), dict(rl=-1), dict(qh=-1),
               dict(qo=0), dict(q=0), dict(rope=0), dict(qh=0)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    assert call(t=1 << 31) == bd.BD_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(q=ODD), dict(k=ODD), dict(rope=ODD), dict(qo=ODD), dict(pos=A + 2), dict(table=A + 1), dict(seq=A + 1)):
        assert call(**kw) == bd.BD_ERR_MISALIGNED, kw
    assert call(t=0, k=0, v=0, pos=0) == bd.BD_OK


def test_kv_read(lib):
    def call(c=cache(), table=A, ns=2, mp=4, off=A, total=10, ko=A, vo=A):
        return lib.bd_kv_read(None if c is None else ctypes.byref(c), table, ns, mp, off, total, ko, vo, None)
    for c, status in BAD_CACHES:
        assert call(c=c) == status
    for kw in (dict(table=0), dict(off=0), dict(ko=0), dict(vo=0), dict(total=-1), dict(ns=-1)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    assert call(total=1 << 31) == bd.BD_ERR_UNSUPPORTED_SHAPE
    assert call(ko=ODD) == bd.BD_ERR_MISALIGNED and call(off=A + 2) == bd.BD_ERR_MISALIGNED
    assert call(total=0, ko=0, vo=0) == bd.BD_OK and call(ns=0, table=0) == bd.BD_OK


def test_attention(lib):
    def call(c=cache(), q=A, qh=4, table=A, lens=A, ns=2, mp=4, scale=1.0, window=0, out=A, lse=A, ws=A, wb=1 << 40):
        return lib.bd_attention_decode(None if c is None else ctypes.byref(c), q, qh, table, lens, ns, mp, scale, window, out, lse,
                                       ws, wb, None)
    for c, status in BAD_CACHES:
        assert call(c=c) == status
    for kw in (dict(q=0), dict(table=0), dict(lens=0), dict(out=0), dict(ns=-1), dict(mp=-1), dict(qh=0), dict(window=-1),
               dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    assert call(qh=5) == bd.BD_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(q=ODD), dict(out=ODD), dict(lens=A + 1), dict(table=A + 2), dict(lse=A + 2)):
        assert call(**kw) == bd.BD_ERR_MISALIGNED, kw
    assert call(ws=0) == bd.BD_ERR_WORKSPACE and call(ws=A + 16) == bd.BD_ERR_WORKSPACE
    assert call(ns=0, q=0, table=0, lens=0, out=0, ws=0) == bd.BD_OK
    for c, _ in BAD_CACHES:
        assert lib.bd_attention_workspace_size(None if c is None else ctypes.byref(c), 1, 4) == 0


def test_sample(lib):
    def call(x=A, lt=0, m=2, v=100, t=A, k=A, p=A, lo=A, g=A, ids=A, lp=A):
        return lib.bd_sample(x, lt, m, v, t, k, p, lo, g, ids, lp, None)
    for kw in (dict(x=0), dict(g=0), dict(ids=0), dict(lt=2), dict(m=-1), dict(v=0)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    assert call(v=bd.BD_SAMPLE_MAX_VOCAB + 1) == bd.BD_ERR_UNSUPPORTED_SHAPE
    assert call(m=1 << 30) == bd.BD_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(x=ODD), dict(g=ODD), dict(t=A + 1), dict(k=A + 2), dict(p=A + 1), dict(lo=A + 3), dict(ids=A + 1), dict(lp=A + 2)):
        assert call(**kw) == bd.BD_ERR_MISALIGNED, kw
    assert call(m=0, x=0, g=0, ids=0) == bd.BD_OK
