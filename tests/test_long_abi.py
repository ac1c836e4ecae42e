"""The long-context entry points refuse bad arguments before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from bit_delta_tenant_gb300 import bitdelta as bd
from bit_delta_tenant_gb300 import build as bd_build
from test_step_abi import BAD_CACHES, A, ODD, cache

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    bd_build.build()
    return bd.load_library()


def four(**kw):
    return cache(**{**dict(kv_type=2, k_scale=A, v_scale=A), **kw})


def ref(c):
    return None if c is None else ctypes.byref(c)


def test_four_bit_caches(lib):
    def status(c):
        return lib.bd_kv_read(ref(c), A, 2, 4, A, 0, 0, 0, None)
    assert status(four()) == bd.BD_OK and status(four(head_dim=128)) == bd.BD_OK
    for kw, want in ((dict(k_scale=0), bd.BD_ERR_INVALID_ARG), (dict(v_scale=0), bd.BD_ERR_INVALID_ARG), (dict(kv_type=3), bd.BD_ERR_INVALID_ARG),
                     (dict(kv_type=-1), bd.BD_ERR_INVALID_ARG), (dict(head_dim=32), bd.BD_ERR_UNSUPPORTED_SHAPE), (dict(k_scale=ODD), bd.BD_ERR_MISALIGNED)):
        assert status(four(**kw)) == want, kw


def test_kv_append_rotary(lib):
    def call(c=four(), q=A, qh=4, k=A, v=A, t=3, seq=A, pos=A, table=A, ns=2, mp=4, rope=A, rl=64, rd=64, lay=0, qo=A):
        return lib.bd_kv_append_rotary(ref(c), q, qh, k, v, t, seq, pos, table, ns, mp, rope, rl, rd, lay, qo, None)
    for c, status in BAD_CACHES:
        assert call(c=c) == status
    for kw in (dict(k=0), dict(pos=0), dict(t=-1), dict(rl=-1), dict(qo=0), dict(q=0), dict(rope=0), dict(lay=2), dict(lay=-1)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    for kw in (dict(rd=0), dict(rd=8), dict(rd=40), dict(rd=80), dict(rd=-16)):
        assert call(**kw) == bd.BD_ERR_UNSUPPORTED_SHAPE, kw
    assert call(rope=ODD) == bd.BD_ERR_MISALIGNED
    assert call(t=0, rd=16, lay=1) == bd.BD_OK and call(t=0, q=0, qo=0, rope=0, rd=0, lay=7) == bd.BD_OK


def test_rotary_table(lib):
    def call(t=A, n=0, dim=64, base=1e4, factor=1.0, original=0.0, low=1.0, high=4.0, amp=1.0):
        return lib.bd_rotary_table(t, n, dim, base, factor, original, low, high, amp, None)
    assert call() == bd.BD_OK and call(t=0) == bd.BD_OK
    for kw in (dict(n=-1), dict(t=0, n=4), dict(dim=0), dict(base=0.0), dict(base=-1.0), dict(base=NAN), dict(base=INF), dict(factor=0.0), dict(factor=-2.0),
               dict(factor=NAN), dict(original=-1.0), dict(original=INF), dict(high=1.0), dict(low=NAN), dict(amp=INF), dict(amp=NAN),
               dict(base=1e-308, dim=256, factor=1e-300)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    for kw in (dict(dim=63), dict(dim=bd.BD_ROTARY_MAX_DIM + 2), dict(n=1 << 31)):
        assert call(**kw) == bd.BD_ERR_UNSUPPORTED_SHAPE, kw
    assert call(t=ODD) == bd.BD_ERR_MISALIGNED


def rule(**kw):
    return bd.ScoreRule(**{**dict(scale=1.0, cap=0.0, slopes=0, first=0, prefix=0, window=0, reserved=0), **kw})


BAD_RULES = [None] + [rule(**kw) for kw in (dict(scale=NAN), dict(scale=INF), dict(cap=-1.0), dict(cap=NAN), dict(cap=INF), dict(cap=1e-40), dict(cap=3e38), dict(window=-1), dict(reserved=1))]
ODD_RULES = [rule(slopes=A + 2), rule(first=A + 1), rule(prefix=A + 3)]


def test_attention_decode_scored(lib):
    def call(c=four(), q=A, qh=4, table=A, lens=A, ns=2, mp=4, r=rule(), out=A, lse=A, ws=A, wb=1 << 40):
        return lib.bd_attention_decode_scored(ref(c), q, qh, table, lens, ns, mp, ref(r), out, lse, ws, wb, None)
    for c, status in BAD_CACHES:
        assert call(c=c) == status
    for r in BAD_RULES:
        assert call(r=r) == bd.BD_ERR_INVALID_ARG
    for r in ODD_RULES:
        assert call(r=r) == bd.BD_ERR_MISALIGNED
    for kw in (dict(q=0), dict(table=0), dict(lens=0), dict(out=0), dict(ns=-1), dict(mp=-1), dict(qh=0)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    assert call(qh=5) == bd.BD_ERR_UNSUPPORTED_SHAPE
    assert call(ws=0) == bd.BD_ERR_WORKSPACE and call(ws=A + 16) == bd.BD_ERR_WORKSPACE
    assert call(ns=0, q=0, table=0, lens=0, out=0, ws=0) == bd.BD_OK


def test_attention_prompt(lib):
    def call(c=four(), q=A, qh=4, off=A, total=5, table=A, lens=A, ns=2, mp=4, r=rule(), out=A, lse=A, ws=A, wb=1 << 40):
        return lib.bd_attention_prompt(ref(c), q, qh, off, total, table, lens, ns, mp, ref(r), out, lse, ws, wb, None)
    for c, status in BAD_CACHES:
        assert call(c=c) == status
        assert lib.bd_attention_prompt_workspace_size(ref(c), 4) == 0
    for r in BAD_RULES:
        assert call(r=r) == bd.BD_ERR_INVALID_ARG
    for r in ODD_RULES:
        assert call(r=r) == bd.BD_ERR_MISALIGNED
    for kw in (dict(q=0), dict(off=0), dict(table=0), dict(lens=0), dict(out=0), dict(ns=-1), dict(mp=-1), dict(total=-1), dict(qh=0)):
        assert call(**kw) == bd.BD_ERR_INVALID_ARG, kw
    assert call(qh=5) == bd.BD_ERR_UNSUPPORTED_SHAPE and call(total=1 << 31) == bd.BD_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(q=ODD), dict(out=ODD), dict(lens=A + 1), dict(off=A + 2), dict(table=A + 2), dict(lse=A + 2)):
        assert call(**kw) == bd.BD_ERR_MISALIGNED, kw
    assert call(ws=0) == bd.BD_ERR_WORKSPACE and call(ws=A + 16) == bd.BD_ERR_WORKSPACE
    assert call(ns=0, q=0, off=0, table=0, lens=0, out=0, ws=0) == bd.BD_OK
    assert call(total=0, q=0, off=0, table=0, lens=0, out=0, ws=0) == bd.BD_OK
