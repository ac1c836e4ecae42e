"""bd_sample where its shorter ways to an answer do not suffice.

top-p looks for the best draw before it knows the prefix's end: noise here favours tokens beyond
that end, at it, or none of those before it.  An unfiltered row is scored before its largest logit
is known: scores here lie within a rounding of each other, or noise and logits at the end of their range.
Bounds as in test_gpu_sample.py."""
import numpy as np
import pytest
import torch

from test_gpu_sample import DTYPES, check, gumbel, logits

pytestmark = pytest.mark.gpu


def places(x):
    """Each token's place in the order (logit descending, index ascending)."""
    order = np.argsort(-x.float().numpy().astype(np.float64), axis=1, kind="stable")
    place = np.empty_like(order)
    np.put_along_axis(place, order, np.arange(order.shape[1])[None, :].repeat(order.shape[0], 0), 1)
    return place


def prefix_ends(x, p, t):
    xf = np.sort(x.float().numpy().astype(np.float64), axis=1)[:, ::-1]
    w = np.exp((xf - xf[:, :1]) / t)
    mass = np.cumsum(w, 1)
    return (mass - w < p * mass[:, -1:]).sum(1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,vocab", [(3, 9001), (40, 5003), (3, 60000)])
@pytest.mark.parametrize("p,t", [(0.02, 1.0), (0.5, 0.4), (0.9, 1.0), (0.97, 8.0)])
@pytest.mark.parametrize("favoured", ["beyond", "at the end", "before", "random"])
def test_top_p_with_noise_that_favours(dtype, m, vocab, p, t, favoured):
    x, g = logits(m, vocab, vocab + m, dtype), gumbel(m, vocab, vocab)
    place, end = places(x), prefix_ends(x, p, t)[:, None]
    lift = {"beyond": place >= end, "at the end": abs(place - end) < 40, "before": place < end,
            "random": np.random.default_rng(1).random((m, vocab)) < 0.01}[favoured]
    g = np.where(lift, g + np.float32(40), g).astype(np.float32)
    check(x, g, p=p, t=t, rows=range(0, m, 3))
    check(x, g, p=p, t=t, low=0.2, rows=range(0, m, 3))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("p", [0.3, 0.9])
def test_top_p_with_no_score_before_the_end(dtype, p):
    x, g = logits(4, 20001, 3, dtype), gumbel(4, 20001, 5)
    place, end = places(x), prefix_ends(x, p, 1.0)[:, None]
    g[:2] = np.where(place < end, -np.inf, g)[:2]
    g[2:] = np.where(place < end, np.nan, g)[2:]
    check(x, g, p=p)


@pytest.mark.parametrize("dtype", DTYPES)
def test_top_p_of_peaked_rows(dtype):
    """One token with nearly all of the weight, or a few alike: the prefix ends in the first bin."""
    v = 30000
    x, g = logits(6, v, 8, dtype, spread=1.0), gumbel(6, v, 9)
    x[0, 777] = 40.0
    x[1, 29999] = 14.0
    x[2, ::1000] = 30.0
    x[3, :3] = 20.0
    x[4] = 1.5
    x[5, :15000], x[5, 15000:] = 2.0, -3.0
    for p in (0.05, 0.5, 0.9, 0.999):
        check(x, g, p=p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,vocab", [(2, 10007), (300, 4099)])
def test_unfiltered_scores_a_rounding_apart(dtype, m, vocab):
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy((rng.integers(0, 4, (m, vocab)) * 2.0 ** -6 + 8).astype(np.float32)).to(dtype)
    g = (rng.integers(0, 8, (m, vocab)) * 2.0 ** -22 + 3).astype(np.float32)
    rows = range(0, m, max(1, m // 12))
    check(x, g, rows=rows)
    check(x, g, t=1e-3, rows=rows)
    check(x, g, t=1e4, rows=rows)
    check(x, np.zeros_like(g), rows=rows)
    check(torch.full_like(x, -7.25), g, rows=rows)


@pytest.mark.parametrize("dtype", DTYPES)
def test_unfiltered_at_the_end_of_the_range(dtype):
    v = 12345
    x, g = logits(8, v, 2, dtype), gumbel(8, v, 3)
    g[0] *= np.float32(1e30)
    g[1, 100], g[1, 9000] = np.inf, np.inf
    g[2, ::2] = np.nan
    g[3] = -np.inf
    x[4] *= 1e30
    x[5, 5::7] = float("nan")
    x[6, 4000] = float("inf")
    x[7] = -3e38
    check(x, g)
    check(x, g, t=1e-30)
    check(x, g, t=1e30)
