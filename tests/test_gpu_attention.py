"""bd_attention_decode on the GPU against the definition in 64 bits.

Bounds.  A score is added up in 8 tensor-core steps of 16 products whose sums may be truncated:
within 2^-19 of scale * sum |q k|, so a weight is within twice that (numerator and sum), plus 2^-17 of
the split weights, 2^-21 of exp2 and the scale's rounding, and up to 128 accumulation steps of 2^-23 in the
output: (2^-14 + 2^-18 * max_j scale * sum |q k_j|) * sum p |v|.  bf16 rounds to 2^-8 of the value."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import Pool, attention, f64, randn

pytestmark = pytest.mark.gpu


def run(pool, q, lengths=None, window=0, scale=None, ws=None, lse=True, out=None):
    cache = pool.cache() if isinstance(pool, Pool) else pool[0]
    table = torch.from_numpy(pool.table).cuda() if isinstance(pool, Pool) else pool[1]
    n, heads, _ = q.shape
    out = torch.full_like(q, 3.0, device="cuda") if out is None else out
    lse = torch.full((n, heads), 3.0, device="cuda") if lse else None
    if ws is None:
        ws = torch.zeros(bd.bd_attention_workspace_size(cache, n, heads), dtype=torch.uint8, device="cuda")
    lens = torch.tensor(pool.lengths if lengths is None else lengths, dtype=torch.int32).cuda()
    bd.bd_attention_decode(cache, q.cuda(), table, lens, out, ws, scale=scale, window=window, lse=lse)
    return out, lse


def check(pool, q, out, lse, window=0, scale=None, lengths=None, seqs=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for i in range(len(pool.lengths)) if seqs is None else seqs:
        n = (pool.lengths if lengths is None else lengths)[i]
        lo = max(0, n - window) if window else 0
        k, v = pool.values("k", i, n)[lo:], pool.values("v", i, n)[lo:]
        ref, ref_lse, mag, big = attention(f64(q[i]), k, v, scale)
        err = np.abs(f64(out[i]) - ref)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -14 + 2.0 ** -18 * big[:, None]) * mag
        assert np.all(err <= tol), (i, n, float((err - tol).max()))
        if n == 0:
            assert (out[i] == 0).all() and (lse is None or torch.isneginf(lse[i]).all())
        elif lse is not None:
            assert np.all(np.abs(f64(lse[i]) - ref_lse) <= 2.0 ** -19 * (np.abs(ref_lse) + 16) + 2.0 ** -18 * big), (i, n)


HEADS = [(32, 8), (4, 4), (8, 1), (1, 1), (12, 1), (16, 1), (48, 2), (40, 2), (7, 7), (9, 3)]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", HEADS)
def test_heads_and_lengths(kv, dim, q_heads, kv_heads):
    """Lengths around the tile (16), the block (64), a page and nothing at all; slots no token uses hold NaN."""
    lengths = [1, 0, 15, 16, 17, 63, 64, 65, 0, 200, 129, 2]
    pool = Pool(lengths, kv_heads, dim, 32, kv, seed=q_heads + dim, junk=0x7F if kv == "e4m3" else float("nan"))
    q = randn((len(lengths), q_heads, dim), 9, 2.0).bfloat16()
    out, lse = run(pool, q)
    check(pool, q, out, lse)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 48, 64, 1024])
def test_pages_and_long_splits(kv, page):
    lengths = [4099, 1, 1000, 0, 2500]
    pool = Pool(lengths, 2, 128, page, kv, seed=page)
    q = randn((5, 8, 128), 9, 2.0).bfloat16()
    out, lse = run(pool, q)
    check(pool, q, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 15, 16, 64, 100, 5000])
def test_window_reads_nothing_before_it(kv, window):
    """Pages wholly before the window have no valid id; older keys in the window's first page hold NaN."""
    lengths = [1, 90, 128, 300, 1000, 0, 64]
    pool = Pool(lengths, 2, 64, 16, kv, seed=window)
    for i, n in enumerate(lengths):
        lo = max(0, n - window)
        for t in range(lo // 16 * 16, lo):
            if kv == "bf16":
                pool.k[pool.table[i, t // 16], :, t % 16] = float("inf")
                pool.v[pool.table[i, t // 16], :, t % 16] = float("nan")
            else:
                pool.k.view(torch.uint8)[pool.table[i, t // 16], :, t % 16] = 0x7F
                pool.v.view(torch.uint8)[pool.table[i, t // 16], :, t % 16] = 0x7F
    table = pool.table.copy()
    for i, n in enumerate(lengths):
        table[i, : max(0, n - window) // 16] = -1
    q = randn((len(lengths), 6, 64), 9, 2.0).bfloat16()
    out, lse = run((pool.cache(), torch.from_numpy(table).cuda()), q, lengths, window=window)
    check(pool, q, out, lse, window=window)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
def test_scales_flat_and_peaked(kv, scale):
    pool = Pool([777, 30], 2, 64, 16, kv, seed=5)
    q = randn((2, 8, 64), 9, 2.0).bfloat16()
    out, lse = run(pool, q, scale=scale)
    check(pool, q, out, lse, scale=scale)


def test_large_and_small_magnitudes():
    """8-bit keys and values whose scales differ by many powers of two between tokens; queries far from 1."""
    pool = Pool([300, 300, 300], 2, 64, 16, "e4m3", seed=6)
    rng = np.random.default_rng(0)
    for s in (pool.k_scale, pool.v_scale):
        s.copy_(torch.from_numpy(rng.integers(127 - 14, 127 - 4, s.shape).astype(np.uint8)))
    pool.v_scale[0] = 67  # nearly nothing beside the others
    q = randn((3, 8, 64), 9).bfloat16()
    q[0] *= 2.0 ** -70
    q[1, :4] *= 2.0 ** 12
    q[1, 4:] *= 2.0 ** -20
    q[2, 1] = 0
    out, lse = run(pool, q, scale=2.0 ** -3)
    check(pool, q, out, lse, scale=2.0 ** -3, seqs=[0, 2])
    # the first heads of the second sequence see scores up to thousands: their bound still holds
    check(pool, q, out, lse, scale=2.0 ** -3, seqs=[1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_bad_query_head_stays_alone(kv):
    pool = Pool([100], 2, 64, 16, kv, seed=5)
    q = randn((1, 8, 64), 9).bfloat16()
    bad = q.clone()
    bad[0, 2, 7] = float("nan")
    a, _ = run(pool, q)
    b, _ = run(pool, bad)
    assert torch.isnan(b[0, 2]).all()
    keep = [0, 1, 3, 4, 5, 6, 7]
    assert torch.equal(a[0, keep], b[0, keep])


def test_repeats_are_identical_and_one_workspace_serves_every_batch():
    big = Pool([3000, 5, 700, 0, 64] * 4, 4, 128, 16, "e4m3", seed=2)
    small = Pool([900], 2, 64, 32, "bf16", seed=3)
    wide = Pool([33] * 300, 1, 64, 16, "bf16", seed=4)
    qs = [randn((len(p.lengths), 4 * p.kv_heads, p.dim), 1).bfloat16() for p in (big, small, wide)]
    need = max(bd.bd_attention_workspace_size(p.cache(), len(p.lengths), 4 * p.kv_heads) for p in (big, small, wide))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = [run(p, q, ws=ws) for p, q in zip((big, small, wide), qs)]
    for p, q, (out, lse) in zip((big, small, wide), qs, first):
        check(p, q, out, lse, seqs=range(min(5, len(p.lengths))))
    for _ in range(3):
        for p, q, (out, lse) in zip((wide, big, small), (qs[2], qs[0], qs[1]), (first[2], first[0], first[1])):
            again = run(p, q, ws=ws)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_many_sequences():
    """More sequences than a CTA has threads, most of them empty."""
    rng = np.random.default_rng(1)
    lengths = [int(n) for n in np.where(rng.random(700) < 0.7, 0, rng.integers(1, 90, 700))]
    pool = Pool(lengths, 1, 64, 16, "bf16", seed=2)
    q = randn((700, 2, 64), 1).bfloat16()
    out, lse = run(pool, q)
    check(pool, q, out, lse)


def test_all_empty_and_no_sequences():
    pool = Pool([0, 0, 0], 2, 64, 16, "bf16", seed=2)
    q = randn((3, 4, 64), 1).bfloat16()
    out, lse = run(pool, q)
    assert (out == 0).all() and torch.isneginf(lse).all()
    cache = pool.cache()
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    bd.bd_attention_decode(cache, e, torch.empty((0, 1), dtype=torch.int32, device="cuda"),
                           torch.empty((0,), dtype=torch.int32, device="cuda"), e.clone(),
                           torch.zeros(256, dtype=torch.uint8, device="cuda"))


def test_bad_pages_and_lengths_flag():
    pool = Pool([100, 60], 1, 64, 16, "bf16", seed=2)
    q = randn((2, 4, 64), 1).bfloat16()
    good = pool.table.copy()
    pool.table[0, 2] = 10 ** 6
    out, _ = run(pool, q)
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    k, v = (np.delete(Pool.values(p, n, 0), np.s_[32:48], 0) for p, n in ((_with(pool, good), "k"), (_with(pool, good), "v")))
    ref, _, mag, big = attention(f64(q[0]), k, v, 64 ** -0.5)
    assert np.all(np.abs(f64(out[0]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -14 + 2.0 ** -18 * big[:, None]) * mag)
    pool.table = good
    check(pool, q, out, None, seqs=[1])
    out, lse = run(pool, q, lengths=[-5, 60])
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    assert (out[0] == 0).all()
    check(pool, q, out, lse, seqs=[1])
    full = Pool([16 * pool.table.shape[1], 60], 1, 64, 16, "bf16", seed=2)
    out, lse = run(full, q, lengths=[16 * full.table.shape[1] + 1, 60])
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    check(full, q, out, lse)


def _with(pool, table):
    pool.table = table
    return pool


def test_in_a_graph_on_another_stream():
    pool = Pool([500, 0, 31], 2, 128, 16, "e4m3", seed=2)
    q = randn((3, 8, 128), 1).bfloat16()
    out, _ = run(pool, q)
    cache, table, qd = pool.cache(), torch.from_numpy(pool.table).cuda(), q.cuda()
    lens, out2 = torch.tensor(pool.lengths, dtype=torch.int32).cuda(), torch.empty_like(out)
    ws = torch.zeros(bd.bd_attention_workspace_size(cache, 3, 8), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            bd.bd_attention_decode(cache, qd, table, lens, out2, ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


def test_refusals():
    pool = Pool([5], 2, 64, 16, "bf16", seed=1)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    cache, table = pool.cache(), torch.from_numpy(pool.table).cuda()
    lens = torch.tensor([5], dtype=torch.int32).cuda()
    ws = torch.zeros(bd.bd_attention_workspace_size(cache, 1, 4), dtype=torch.uint8, device="cuda")
    for args in ((q.float(), table, lens, q.clone()), (q, table, lens.long(), q.clone()), (q, table, lens, q[:, :2]),
                 (q[0], table, lens, q.clone()), (q, table.float(), lens, q.clone()), (q[..., :32], table, lens, q.clone())):
        with pytest.raises(ValueError):
            bd.bd_attention_decode(cache, *args, ws)
    for kw, status in ((dict(workspace=ws[:256]), bd.BD_ERR_WORKSPACE), (dict(window=-1), bd.BD_ERR_INVALID_ARG),
                       (dict(scale=float("nan")), bd.BD_ERR_INVALID_ARG)):
        with pytest.raises(bd.BitDeltaError) as e:
            bd.bd_attention_decode(cache, q, table, lens, q.clone(), **{"workspace": ws, **kw})
        assert e.value.status == status
    odd = torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bd.BitDeltaError) as e:
        bd.bd_attention_decode(cache, odd, table, lens, odd.clone(), ws)
    assert e.value.status == bd.BD_ERR_UNSUPPORTED_SHAPE
