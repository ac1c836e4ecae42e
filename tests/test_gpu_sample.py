"""bd_sample on the GPU against the definition.

z and z + noise are defined down to their roundings, so the drawn token is unique except where
the share p ends: sums of weights are within 2^-20, so the token has to be that of p, of p (1 - 2^-18) or of
p (1 + 2^-18).  logprob: the sum within 2^-20, the logarithm and the subtraction one fp32 rounding each."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import randn, sample

pytestmark = pytest.mark.gpu


def gumbel(m, v, seed):
    u = np.random.default_rng(seed).random((m, v)).clip(1e-7, 1 - 1e-7)
    return (-np.log(-np.log(u))).astype(np.float32)


def draw(x, noise, t=None, k=None, p=None, low=None, logprob=True):
    m = x.shape[0]
    dev = lambda v, d: None if v is None else torch.tensor(np.broadcast_to(np.asarray(v), (m,)).copy(), dtype=d).cuda()  # noqa: E731
    ids = torch.full((m,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((m,), 3.0, device="cuda") if logprob else None
    bd.bd_sample(x.cuda(), torch.from_numpy(noise).cuda(), ids, temperature=dev(t, torch.float32), top_k=dev(k, torch.int32),
                 top_p=dev(p, torch.float32), min_p=dev(low, torch.float32), logprob=lp)
    return ids.cpu().numpy(), None if lp is None else lp.cpu().numpy()


def check(x, noise, t=1.0, k=0, p=1.0, low=0.0, rows=None):
    ids, lp = draw(x, noise, t, k, p, low)
    m = x.shape[0]
    t, k, p, low = (np.broadcast_to(np.asarray(v), (m,)) for v in (t, k, p, low))
    xf = x.float().numpy()
    for r in range(m) if rows is None else rows:
        f = np.float32
        tr, pr, lr = f(t[r]), float(f(p[r])), float(f(low[r]))
        ok = {sample(xf[r], noise[r], tr, k[r], pr * c if pr < 1 else pr, lr) for c in (1, 1 - 2.0 ** -18, 1 + 2.0 ** -18)}
        assert ids[r] in {i for i, _ in ok}, (r, ids[r], ok, t[r], k[r], p[r], low[r])
        ref = next(q for i, q in ok if i == ids[r])
        assert lp[r] == ref or abs(lp[r] - ref) <= 2.0 ** -18 + 2.0 ** -22 * abs(ref), (r, lp[r], ref)


def logits(m, v, seed, dtype, spread=2.5):
    return randn((m, v), seed, spread).to(dtype)


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 1000, 1003, 16384, 16385, 32001, 50000, 128256, 131071, 131072,
                                   200003, 262139, 262144])
def test_vocabularies_with_mixed_settings(dtype, vocab):
    m = 9
    x, g = logits(m, vocab, vocab, dtype), gumbel(m, vocab, vocab)
    check(x, g, t=[1, 0.7, 1.3, 0, 1, 0.9, 2, 1, 0.5], k=[0, 50, 0, 0, 5, 1, 400, 0, 2], p=[1, 1, 0.9, 1, 0.8, 1, 0.95, 1, 0.01],
          low=[0, 0, 0, 0, 0, 0, 0, 0.05, 0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [1, 2, 511, 512, 513, 5000, 19999, 20000, 20001, -3])
@pytest.mark.parametrize("p", [1.0, 0.9])
def test_top_k(dtype, k, p):
    check(logits(3, 20000, k + 9, dtype), gumbel(3, 20000, 1), k=k, p=p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("p", [0.0, -1.0, 1e-6, 0.1, 0.5, 0.9, 0.99, 0.9999, 0.9999999, 1.0, 2.0])
@pytest.mark.parametrize("t", [0.3, 1.0, 30.0])
def test_top_p(dtype, p, t):
    """At t = 30 the whole vocabulary falls into a few bins, which are split again."""
    check(logits(3, 40000, 4, dtype), gumbel(3, 40000, 2), p=p, t=t)


@pytest.mark.parametrize("k,p", [(0, 0.5), (700, 1.0), (3000, 0.5), (1, 1.0), (10000, 0.75), (9, 0.4)])
def test_equal_logits_are_ordered_by_index(k, p):
    x = torch.zeros((2, 10000), dtype=torch.bfloat16)
    x[1, 5000:] = 1.0
    g = np.zeros((2, 10000), np.float32)
    g[:, ::7] = 1.0
    check(x, g, k=k, p=p)
    check(x, gumbel(2, 10000, 3), k=k, p=p)


def test_few_values_many_ties():
    x = (randn((4, 60000), 5).mul(2).round() / 2).bfloat16()
    check(x, gumbel(4, 60000, 6), k=[0, 7000, 100, 30000], p=[0.7, 1.0, 0.9, 0.3])


@pytest.mark.parametrize("dtype", DTYPES)
def test_masks(dtype):
    """-inf, the type's lowest value, NaN, +inf; rows in which nothing, one token or everything is masked."""
    v = 5000
    lowest = torch.finfo(dtype).min
    x = logits(9, v, 8, dtype)
    x[0, 100:] = -float("inf")
    x[1, 100:] = lowest
    x[2] = -float("inf")
    x[3] = lowest
    x[4] = -float("inf")
    x[4, 4321] = -5
    x[5, ::2] = float("nan")
    x[6, 17] = x[6, 4000] = float("inf")
    x[7] = float("nan")
    x[8, 1:] = lowest
    g = gumbel(9, v, 3)
    for kw in (dict(), dict(p=0.9), dict(k=300), dict(k=4000, p=0.5), dict(low=0.1), dict(t=0.0), dict(t=0.25), dict(k=2, p=0.9)):
        check(x, g, **kw)
    ids, lp = draw(x, g)
    assert ids[2] == -1 and ids[7] == -1 and np.isneginf(lp[[2, 7]]).all()
    assert ids[4] == 4321 and ids[0] < 100 and ids[1] < 100 and ids[8] == 0 and ids[6] in (17, 4000) and ids[5] % 2 == 1


def test_odd_settings_and_noise():
    v = 3000
    x, g = logits(8, v, 9, torch.float32), gumbel(8, v, 4)
    nan, inf = float("nan"), float("inf")
    check(x, g, t=[nan, -1, 1e-30, 1e30, inf, 1e-45, 1, 1])
    check(x, g, p=[nan, 1, 1, 1, 1, 1, 1, 1], low=[nan, 2, 1, -1, 0.999, 0.5, 0.1, 1e-9])
    g[0, 5], g[1, 7:] = nan, -inf
    g[2], g[3] = -inf, nan
    g[4, 2999] = inf
    check(x, g)
    check(x, g, k=1)
    check(x, g, p=0.5)


def test_defaults_and_negative_zero():
    x = torch.tensor([[-0.0, 0.0, -0.0, -1.0]])
    g = np.zeros((1, 4), np.float32)
    ids, _ = draw(x, g)
    assert ids[0] == 0
    ids, lp = draw(x, np.array([[0, 0.5, 0.5, 0]], np.float32), logprob=False)
    assert ids[0] == 1 and lp is None
    ids, _ = draw(x, np.array([[0, 0.5, 0.5, 0]], np.float32), k=1)
    assert ids[0] == 0


def test_frequencies_follow_the_kept_weights():
    """20000 draws of one row: each kept token's count within 5 standard deviations, no other token ever."""
    v, n = 300, 20000
    row = randn((1, v), 3, 2.0)
    x = row.expand(n, v).contiguous()
    ids, _ = draw(x, gumbel(n, v, 7), t=0.8, k=40, p=0.9, low=0.01)
    z = (row[0].double().numpy() - float(row.max())) / 0.8
    w = np.exp(z)
    order = np.argsort(-w)[:40]
    mass = np.cumsum(w[order])
    order = order[np.concatenate([[True], mass[:-1] < 0.9 * mass[-1]])]
    order = order[w[order] >= 0.01]
    pr = np.zeros(v)
    pr[order] = w[order] / w[order].sum()
    count = np.bincount(ids, minlength=v)
    assert np.all(np.abs(count - n * pr) <= 5 * np.sqrt(n * pr * (1 - pr)) + 1e-9)


def test_many_rows_repeat_identically():
    x, g = logits(300, 40000, 3, torch.float32), gumbel(300, 40000, 5)
    kw = dict(t=1.5, k=np.arange(300) * 7 % 1000, p=0.9)
    a, b = draw(x, g, **kw), draw(x, g, **kw)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("t", [1.0, 300.0])
def test_more_rows_than_the_gpu_holds(t):
    """One CTA per row: at t = 300 all 70001 tokens of it lie in a few bins."""
    m, v = 700, 70001
    x = logits(m, v, 6, torch.bfloat16)
    u = torch.rand((m, v), generator=torch.Generator().manual_seed(1)).clamp_(1e-7, 1 - 1e-7)
    g = u.log_().neg_().log_().neg_().numpy()
    k = np.where(np.arange(m) % 3 == 0, 30000, 0)
    p = np.where(np.arange(m) % 3 == 1, 0.9, 1.0)
    check(x, g, t=t, k=k, p=p, rows=[0, 1, 2, 349, 350, 697, 699])


def test_no_rows_and_refusals():
    e = torch.empty((0, 100), device="cuda")
    i32 = torch.empty((0,), dtype=torch.int32, device="cuda")
    bd.bd_sample(e, e.clone(), i32)
    x = torch.zeros((2, 100), device="cuda")
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    for a, kw in (((x, x[:1], ids), {}), ((x, x, ids.long()), {}), ((x.half(), x, ids), {}), ((x, x.bfloat16(), ids), {}),
                  ((x, x, ids), dict(top_k=ids.float())), ((x, x, ids), dict(temperature=ids)), ((x, x, ids), dict(top_p=x[0])),
                  ((x.t().contiguous().t(), x, ids), {})):
        with pytest.raises(ValueError):
            bd.bd_sample(*a, **kw)
    big = torch.zeros((1, bd.BD_SAMPLE_MAX_VOCAB + 1), device="cuda")
    with pytest.raises(bd.BitDeltaError) as err:
        bd.bd_sample(big, big.clone(), ids[:1])
    assert err.value.status == bd.BD_ERR_UNSUPPORTED_SHAPE
