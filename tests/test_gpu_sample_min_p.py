"""min-p of bd_sample at its very edge: the last token that stays and the first that does not, in rows whose threshold
logit is near zero beside a large maximum, where the threshold's own rounding is larger than the logit.

The tokens' weights lie 2^-21 of themselves above and below min_p: a weight is exp of an fp32 z, and expf is off by
two units in the last place at most, 2^-22."""
import numpy as np
import pytest
import torch

from test_gpu_sample import check

pytestmark = pytest.mark.gpu
F = np.float32


def weight(x, top, t):
    z = ((x - top).astype(F) * (F(1) / t).astype(F)).astype(F)
    return np.exp(z.astype(np.float64))


def edges(top, t, low):
    """Per row the smallest logit of weight >= low (1 + 2^-21) and the largest of weight <= low (1 - 2^-21), by bisection
    over the bits of fp32 in ascending order."""
    up = lambda x: np.where(x.view(np.int32) < 0, np.int64(-2 ** 31) - x.view(np.int32), x.view(np.int32).astype(np.int64))  # noqa: E731
    down = lambda n: np.where(n < 0, np.int64(-2 ** 31) - n, n).astype(np.int32).view(F)  # noqa: E731
    out = []
    for bound in (low.astype(np.float64) * (1 + 2.0 ** -21), low.astype(np.float64) * (1 - 2.0 ** -21)):
        a, b = up(np.full_like(top, -100)), up(top)
        while np.any(b - a > 1):
            mid = (a + b) // 2
            on = weight(down(mid), top, t) >= bound
            a, b = np.where(on, a, mid), np.where(on, mid, b)
        out.append(b if not out else a)
    return down(out[0]), down(out[1])


@pytest.mark.parametrize("favoured", ["last that stays", "first that does not"])
@pytest.mark.parametrize("offset", [0.0, 0.01, 1.0])
def test_edge(favoured, offset):
    """offset: how far the threshold logit is from zero."""
    m, v = 3000, 240
    rng = np.random.default_rng(1)
    t = rng.uniform(0.3, 3, m).astype(F)
    depth = rng.uniform(1, 30, m)
    top = (depth * t + offset * rng.uniform(-1, 1, m)).astype(F)
    low = np.exp(-depth).astype(F)
    stays, goes = edges(top, t, low)
    assert np.all(stays > goes)
    x = np.full((m, v), -80, F)
    at = rng.integers(8, v // 2, m)
    r = np.arange(m)
    x[r, 3], x[r, at], x[r, at + v // 2] = top, stays, goes
    g = np.zeros((m, v), F)
    g[r, at if favoured == "last that stays" else at + v // 2] = 60
    check(torch.from_numpy(x), g, t=t, low=low)


def test_a_threshold_next_to_zero():
    """A token at 7.2291e-4 whose weight, 1.9826528e-4, is above min_p."""
    x = torch.full((1, 1000), -60.0)
    x[0, 2], x[0, 700] = 16.027365, 7.2291e-4
    g = np.zeros((1, 1000), F)
    g[0, 700] = 60
    check(x, g, t=F(1.8797584), low=F(1.98265e-4))
