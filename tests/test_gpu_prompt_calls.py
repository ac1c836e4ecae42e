"""bd_attention_prompt as it is called: graphs, streams, workspaces, bad indices, rows of no sequence, pools past 32 bits, waits
that run out.  Bounds are test_gpu_prompt's."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool
from step_ref import randn
from test_gpu_prompt import case, check, offsets_of, run

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "e2m1"]


@pytest.mark.parametrize("kv", KINDS)
def test_replayed_with_other_contents(kv):
    """A captured call with what it was captured with, then longer and shorter sequences, other pages, splits and none."""
    cases = [([40, 3, 200], [0, 30, 100]), ([5, 1, 2], [1500, 0, 9]), ([0, 243, 0], [3, 0, 0])]
    pools = [case(kv, 128, 8, 2, new, past, page=16, seed=i) for i, (new, past) in enumerate(cases)]
    n_pages, width = max(p.k.shape[0] for p, _ in pools), max(p.table.shape[1] for p, _ in pools)
    fields = [f for f in ("k", "v", "k_scale", "v_scale") if getattr(pools[0][0], f) is not None]
    held = {f: torch.zeros((n_pages, *getattr(pools[0][0], f).shape[1:]), dtype=getattr(pools[0][0], f).dtype, device="cuda") for f in fields}
    cache = bd.KVCache(**held)
    table = torch.zeros((3, width), dtype=torch.int32, device="cuda")
    q = torch.zeros((243, 8, 128), dtype=torch.bfloat16, device="cuda")
    off, lens = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((243, 8), device="cuda")
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, 8), dtype=torch.uint8, device="cuda")

    def load(i):
        pool, x = pools[i]
        for f in fields:
            held[f].view(torch.uint8)[:getattr(pool, f).shape[0]].copy_(getattr(pool, f).view(torch.uint8))
        table[:, :pool.table.shape[1]].copy_(torch.from_numpy(pool.table))
        q[:x.shape[0]].copy_(x)
        off.copy_(offsets_of(cases[i][0])), lens.copy_(torch.tensor(pool.lengths, dtype=torch.int32))
        out.fill_(7)

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.bd_attention_prompt(cache, q, off, table, lens, out, ws, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.bd_attention_prompt(cache, q, off, table, lens, out, ws, lse=lse)
    for i in (1, 0, 2, 1, 1):
        load(i)
        graph.replay()
        n = sum(cases[i][0])
        check(pools[i][0], pools[i][1], cases[i][0], out[:n], lse[:n])
        assert (out[n:] == 7).all()
    assert bd.bd_get_device_status() == bd.BD_OK


def test_two_streams_with_a_workspace_each():
    a, b = case("bf16", 128, 16, 2, [3, 9], [4000, 100], seed=1), case("e2m1", 128, 16, 2, [6], [3000], seed=2)
    want = run(a[0], a[1], [3, 9]), run(b[0], b[1], [6])
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for (pool, q), new, stream in ((a, [3, 9], streams[0]), (b, [6], streams[1])):
            with torch.cuda.stream(stream):
                got.append(run(pool, q, new))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2]))


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("page", [16, 64])
def test_bad_pages_hide_their_keys(kv, page):
    """A page id out of range: the status says so, its keys count as unseen, other sequences are as they were."""
    new, past = [100, 60], [60, 2000]
    pool, q = case(kv, 128, 4, 2, new, past, page=page, seed=3)
    want, _ = run(pool, q, new)
    table = pool.table.copy()
    table[0, 64 // page] = -7
    out, lse = run(pool, q, new, table=torch.from_numpy(table).cuda())
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    assert torch.equal(out[100:], want[100:])
    lost = np.arange(64, 64 + page)
    rows = list(range(0, 100, 9))
    from long_ref import attention
    from step_ref import f64
    k, v = pool.values("k", 0), pool.values("v", 0)
    for r in rows:
        p = 60 + r
        keep = np.setdiff1d(np.arange(p + 1), lost)
        ref, ref_lse, mag, big = attention(f64(q[r]), k[keep], v[keep], len(keep) - 1, 128 ** -0.5)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -18 * big[:, None]) * mag
        assert np.all(np.abs(f64(out[r]) - ref) <= tol), r
    table[1, 5] = pool.k.shape[0]
    run(pool, q, new, table=torch.from_numpy(table).cuda())
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX


def test_bad_lengths_and_offsets_flag():
    pool, q = case("bf16", 64, 4, 2, [20, 30], [0, 10], page=16, seed=3)
    want, want_lse = run(pool, q, [20, 30])
    # longer than the table: counts as what the table holds; shorter than its rows: the first of them see nothing
    out, lse = run(pool, q, [20, 30], lengths=[5, 40])
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    assert (out[:15] == 0).all() and torch.isneginf(lse[:15]).all() and torch.equal(out[20:], want[20:])
    run(pool, q, [20, 30], lengths=[-1, 40])
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    run(pool, q, [20, 30], lengths=[20, 1000])
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
    for offsets in ([0, 20, 51], [0, -5, 50], [0, 20, 10]):  # past the rows, before them, descending: left out
        out, _ = run(pool, q, [20, 30], offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
        assert bd.bd_get_device_status() == bd.BD_ERR_BAD_INDEX
        assert (out[20:] == 3).all()
    assert bd.bd_get_device_status() == bd.BD_OK
    out, lse = run(pool, q, [20, 30])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_rows_of_no_sequence_stay_as_they_are():
    pool, q = case("e4m3", 64, 4, 2, [20, 30], [0, 10], page=16, seed=3)
    more = torch.cat([q, q[:40]])
    out, lse = run(pool, more, [20, 30])
    check(pool, q, [20, 30], out[:50], lse[:50])
    assert (out[50:] == 3).all() and (lse[50:] == 3).all()


def test_one_workspace_for_caches_of_either_head_dim():
    """Split and whole units in turn, on the workspace of the larger head_dim."""
    cases = [case("bf16", 128, 16, 2, [5], [5000], seed=1), case("bf16", 64, 16, 2, [900], [0], seed=2), case("e2m1", 64, 16, 2, [3], [4000], seed=3),
             case("e4m3", 128, 16, 2, [900], [0], seed=4)]
    want = [run(pool, q, [q.shape[0]]) for pool, q in cases]
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cases[0][0].cache(), 16), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 1, 3, 0, 2, 3, 1):
        got = run(*cases[i], [cases[i][1].shape[0]], ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
    assert bd.bd_get_device_status() == bd.BD_OK


def test_one_workspace_for_prompts_and_single_tokens():
    """A prompt's, used by single tokens' attention in between: many parts of one sequence, whole and split units."""
    cases = [case("bf16", 128, 16, 2, [5], [5000], seed=1), case("e4m3", 64, 16, 2, [900], [0], seed=2)]
    one, q = case("bf16", 128, 32, 2, [1], [40000], seed=3)
    q, cache, table, lens = q.cuda(), one.cache(), torch.from_numpy(one.table).cuda(), torch.tensor(one.lengths, dtype=torch.int32, device="cuda")

    def token(ws):
        out = torch.empty_like(q)
        bd.bd_attention_decode(cache, q, table, lens, out, ws)
        return out

    want = [run(pool, x, [x.shape[0]]) for pool, x in cases]
    first = token(torch.zeros(bd.bd_attention_workspace_size(cache, 1, 32), dtype=torch.uint8, device="cuda"))
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, 32), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 1, 0, 1):
        assert torch.equal(token(ws), first), i
        assert all(torch.equal(a, b) for a, b in zip(run(*cases[i], [cases[i][1].shape[0]], ws=ws), want[i])), i
    assert torch.equal(token(ws), first)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("window", [0x7FFFFFFF, 1 << 40])
def test_the_largest_window_and_no_lse(window):
    """More rows than the sequence is long, whose first positions lie below 0, with a window as wide as there is."""
    pool, q = case("bf16", 64, 4, 2, [20, 30], [0, 10], page=16, seed=3)
    want, _ = run(pool, q, [20, 30], lengths=[5, 40])
    out, _ = run(pool, q, [20, 30], lengths=[5, 40], window=window)
    assert torch.equal(out, want)
    cache = pool.cache()
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, 4), dtype=torch.uint8, device="cuda")
    bd.bd_attention_prompt(cache, q.cuda(), offsets_of([20, 30]), torch.from_numpy(pool.table).cuda(), torch.tensor([5, 40], dtype=torch.int32).cuda(), out.zero_(), ws)
    assert torch.equal(out, want)
    bd.bd_get_device_status()


def test_nothing_cached_and_no_rows():
    pool, q = case("bf16", 64, 4, 2, [5, 3], [0, 0], page=16, seed=3)
    out, lse = run(pool, q, [5, 3], lengths=[0, 0])
    assert (out == 0).all() and torch.isneginf(lse).all()
    bd.bd_get_device_status()
    cache = pool.cache()
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, 4), dtype=torch.uint8, device="cuda")
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    empty = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    bd.bd_attention_prompt(cache, empty, ints(3), ints(2, 4), ints(2), empty.clone(), ws)
    bd.bd_attention_prompt(cache, q.cuda(), ints(1), ints(0, 4), ints(0), torch.empty_like(q, device="cuda"), ws)
    out = torch.full_like(q, 3.0, device="cuda")
    bd.bd_attention_prompt(cache, q.cuda(), offsets_of([5, 3]), ints(2, 0), ints(2), out, ws)  # a table without columns
    assert (out == 0).all()
    bd.bd_get_device_status()


@pytest.mark.parametrize("kv", KINDS)
def test_many_sequences(kv):
    """More sequences than a scan's 32 lanes, most of them of a token or none."""
    rng = np.random.default_rng(4)
    new, past = rng.integers(0, 4, 300).tolist(), rng.integers(0, 40, 300).tolist()
    new[77], new[299] = 150, 9
    pool, q = case(kv, 64, 2, 1, new, past, page=16, seed=7, junk=True)
    out, lse = run(pool, q, new)
    check(pool, q, new, out, lse)


def test_pools_past_32_bits():
    """Pages whose bytes lie past 2^33."""
    heads, page, dim = 64, 1024, 128
    n_pages = 1 + (1 << 27) // (heads * page) + 3
    pool, q = case("e2m1", dim, 64, heads, [70, 2], [50, 1030], page=page, seed=5)
    big = {"k": (n_pages, heads, page, dim // 2), "v": (n_pages, heads, page, dim // 2), "k_scale": (n_pages, heads, page, dim // 16),
           "v_scale": (n_pages, heads, page, dim // 16)}
    held = {}
    used = sorted({int(p) for p in pool.table.ravel() if p >= 0})
    where = {p: n_pages - 1 - i for i, p in enumerate(used)}
    for f, shape in big.items():
        held[f] = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for p, at in where.items():
            held[f][at] = getattr(pool, f)[p].cuda()
    table = torch.tensor([[where.get(int(p), -1) for p in row] for row in pool.table], dtype=torch.int32).cuda()
    cache = bd.KVCache(held["k"], held["v"], held["k_scale"], held["v_scale"])
    want = run(pool, q, [70, 2])

    got = run_held(cache, q, [70, 2], pool.lengths, table)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    out, lse = torch.empty((2, 64, dim), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 64), device="cuda")
    ws = torch.zeros(bd.bd_attention_workspace_size(cache, 2, 64), dtype=torch.uint8, device="cuda")
    lens = torch.tensor(pool.lengths, dtype=torch.int32).cuda()
    last = q[[69, 71]].cuda()
    bd.bd_attention_decode(cache, last, table, lens, out, ws, lse=lse)
    small = torch.empty_like(out)
    bd.bd_attention_decode(pool.cache(), last, torch.from_numpy(pool.table).cuda(), lens, small, ws)
    assert torch.equal(out, small)
    rows = [torch.empty((sum(pool.lengths), heads, dim), dtype=torch.bfloat16, device="cuda") for _ in "kvkv"]
    bd.bd_kv_read(cache, table, offsets_of(pool.lengths), rows[0], rows[1])
    bd.bd_kv_read(pool.cache(), torch.from_numpy(pool.table).cuda(), offsets_of(pool.lengths), rows[2], rows[3])
    assert torch.equal(rows[0], rows[2]) and torch.equal(rows[1], rows[3])


def run_held(cache, q, new, lengths, table):
    out, lse = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 3.0, device="cuda")
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, q.shape[1]), dtype=torch.uint8, device="cuda")
    bd.bd_attention_prompt(cache, q.cuda(), offsets_of(new), table, torch.tensor(lengths, dtype=torch.int32).cuda(), out, ws, lse=lse)
    return out, lse


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("new,past", [([300], [0]), ([4], [3000])])
def test_waits_that_run_out_are_reported(kv, new, past):
    """With no time to wait at all the kernel gives up, says so and leaves the next call sound, on the same workspace."""
    pool, q = case(kv, 128, 8, 2, new, past, seed=3)
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(pool.cache(), 8), dtype=torch.uint8, device="cuda")
    want = run(pool, q, new, ws=ws)
    before = bd.bd_set_wait_limit_ns(0)
    try:
        run(pool, q, new, ws=ws)
        assert bd.bd_get_device_status() == bd.BD_ERR_DEVICE_TIMEOUT
    finally:
        bd.bd_set_wait_limit_ns(before)
    again = run(pool, q, new, ws=ws)
    assert bd.bd_get_device_status() == bd.BD_OK
    assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_refusals():
    pool, q = case("bf16", 64, 4, 2, [5], [0], page=16, seed=3)
    cache, table = pool.cache(), torch.from_numpy(pool.table).cuda()
    off, lens, q = offsets_of([5]), torch.tensor([5], dtype=torch.int32).cuda(), q.cuda()
    out = torch.empty_like(q)
    ws = torch.zeros(bd.bd_attention_prompt_workspace_size(cache, 4), dtype=torch.uint8, device="cuda")
    good = dict(q=q, offsets=off, page_table=table, lengths=lens, out=out, workspace=ws)
    f32 = torch.zeros(4, device="cuda")
    for kw in (dict(q=q.float()), dict(q=q[:, :2]), dict(offsets=off.long()), dict(offsets=off[:1]), dict(page_table=table[0]), dict(lengths=lens.cpu()),
               dict(out=out[:4]), dict(lse=f32), dict(slopes=f32[:3]), dict(slopes=f32.double()), dict(first=lens), dict(prefix=off),
               dict(out=out.transpose(0, 1)), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            bd.bd_attention_prompt(cache, **{**good, **kw})
    for kw, status in ((dict(cap=-1.0), bd.BD_ERR_INVALID_ARG), (dict(scale=float("nan")), bd.BD_ERR_INVALID_ARG), (dict(window=-2), bd.BD_ERR_INVALID_ARG),
                       (dict(workspace=ws[:1024]), bd.BD_ERR_WORKSPACE)):
        with pytest.raises(bd.BitDeltaError) as e:
            bd.bd_attention_prompt(cache, **{**good, **kw})
        assert e.value.status == status
    with pytest.raises(ValueError):
        bd.KVCache(*[torch.zeros((2, 1, 16, 32), dtype=torch.uint8, device="cuda") for _ in "kv"])
    with pytest.raises(ValueError):
        bd.KVCache(*[torch.zeros((2, 1, 16, n), dtype=torch.uint8, device="cuda") for n in (32, 32, 4, 2)])
    assert bd.bd_get_device_status() == bd.BD_OK
