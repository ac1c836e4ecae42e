"""Rotary positions: the table against the definition in 64 bits, and pairs of either layout on part of a head as they are
written to every type of cache.

The table's bound is the declared one, 2^-22 of the amplitude, plus fp32's rounding, 2^-24 of the value.  Rotated values are
defined to the bit (each product and sum in fp32, one rounding to the cache's type), so they are equal."""
import math

import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool, four_bits
from step_ref import quantised, randn

pytestmark = pytest.mark.gpu


def table(positions, dim, base=1e4, factor=1.0, original=0.0, low=1.0, high=4.0, amplitude=1.0, rows=None):
    f = base ** (-2.0 * np.arange(dim // 2) / dim)
    g = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
    f = f * (g + (1 - g) / factor)
    a = (np.arange(positions) if rows is None else rows)[:, None] * f
    return amplitude * np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("positions,dim", [(1, 2), (7, 6), (1000, 64), (4097, 128), (33, 256), (5, 10)])
@pytest.mark.parametrize("kw", [dict(), dict(base=5e5, factor=8.0, original=8192.0), dict(factor=4.0), dict(factor=16.0, original=4096.0, low=1.0,
                         high=32.0, amplitude=1.3), dict(base=0.5, amplitude=-2.0)], ids=str)
def test_table(positions, dim, kw):
    t = torch.full((positions, dim), 9.0, device="cuda")
    bd.bd_rotary_table(t, **{"base": 1e4, **kw})
    want = table(positions, dim, **kw)
    amp = abs(kw.get("amplitude", 1.0))
    assert np.all(np.abs(t.cpu().double().numpy() - want) <= amp * 2.0 ** -22 + 2.0 ** -24 * np.abs(want))


def test_far_positions():
    """Two million positions; frequencies within 2^-52 turn a far angle by less than 2^-30."""
    n = 1 << 21
    t = torch.empty((n, 16), device="cuda")
    bd.bd_rotary_table(t, 1e4)
    rows = np.array([0, 1, 12345, n // 2 + 1, n - 1])
    assert np.all(np.abs(t[torch.from_numpy(rows).cuda()].cpu().double().numpy() - table(n, 16, rows=rows)) <= 2.0 ** -22 + 2.0 ** -24)


def test_table_refusals():
    t = torch.empty((4, 16), device="cuda")
    for kw in (dict(base=0.0), dict(base=float("nan")), dict(base=1e4, factor=0.0), dict(base=1e4, original=-1.0),
               dict(base=1e4, low=4.0, high=4.0), dict(base=1e4, amplitude=float("inf"))):
        with pytest.raises(bd.BitDeltaError) as e:
            bd.bd_rotary_table(t, **kw)
        assert e.value.status == bd.BD_ERR_INVALID_ARG
    with pytest.raises(bd.BitDeltaError) as e:
        bd.bd_rotary_table(torch.empty((4, 15), device="cuda"), 1e4)
    assert e.value.status == bd.BD_ERR_UNSUPPORTED_SHAPE
    with pytest.raises(ValueError):
        bd.bd_rotary_table(torch.empty((4, 16), device="cuda", dtype=torch.float64), 1e4)
    bd.bd_rotary_table(torch.empty((0, 16), device="cuda"), 1e4)


def rotated(x, rope, interleaved):
    """x [t, heads, dim] and rope [t, n] in fp32, each operation rounded."""
    n = rope.shape[1]
    c, s = rope[:, None, :n // 2], rope[:, None, n // 2:]
    y = x.float().clone()
    one = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    a, b = y[..., one[0]].clone(), y[..., one[1]].clone()
    y[..., one[0]], y[..., one[1]] = a * c - b * s, b * c + a * s
    return y


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,part,q_heads,kv_heads", [(64, 64, 5, 3), (64, 16, 7, 1), (64, 48, 32, 8), (128, 128, 3, 2), (128, 32, 9, 9),
                                                       (128, 112, 32, 8), (128, 80, 1, 40)])
def test_parts_and_layouts(kv, interleaved, dim, part, q_heads, kv_heads):
    new = [1, 5, 0, 20]
    pool = Pool([30, 40, 3, 50], kv_heads, dim, 16, kv, seed=part)
    t = sum(new)
    seq = np.repeat(np.arange(4), new)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(pool.lengths, new)])
    pos[3] = -1  # a padded token
    rope = torch.from_numpy(table(64, part).astype(np.float32))
    q, k, v = (randn((t, h, dim), 3 + i, 1.5).bfloat16() for i, h in enumerate((q_heads, kv_heads, kv_heads)))
    v[2, 0, :20] = 0.0
    cache = pool.cache()
    before = [x.clone() for x in (cache.k, cache.v) + (() if kv == "bf16" else (cache.k_scale, cache.v_scale))]
    qd = q.cuda()
    bd.bd_kv_append_rotary(cache, qd, k.cuda(), v.cuda(), torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(pool.table).cuda(), rope.cuda(),
                           qd, seq_ids=torch.from_numpy(seq.astype(np.int32)).cuda(), interleaved=interleaved)
    live = pos >= 0
    turned = rope[torch.from_numpy(np.maximum(pos, 0))]
    want_q = torch.where(torch.from_numpy(live)[:, None, None], rotated(q, turned, interleaved).bfloat16(), q)
    assert torch.equal(qd.cpu(), want_q)
    page, slot = pool.table[seq, np.maximum(pos, 0) // 16][live], (np.maximum(pos, 0) % 16)[live]
    for i, (name, x) in enumerate((("k", rotated(k, turned, interleaved)), ("v", v.float()))):
        x, scale = x[torch.from_numpy(live)], None
        x, scale = (x.bfloat16(), None) if kv == "bf16" else quantised(x) if kv == "e4m3" else four_bits(x)
        pool_want = before[i].cpu().clone()
        raw = (lambda y: y.view(torch.uint8)) if kv == "e4m3" else (lambda y: y)
        raw(pool_want)[page, :, slot] = raw(x)
        assert torch.equal(raw(getattr(cache, name).cpu()), raw(pool_want)), name
        if scale is not None:
            want = before[2 + i].cpu().clone()
            want[page, :, slot] = scale
            assert torch.equal(getattr(cache, name + "_scale").cpu(), want), name
    assert bd.bd_get_device_status() == bd.BD_OK
