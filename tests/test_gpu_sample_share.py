"""top-p of bd_sample where the prefix is a few heavy tokens and p lies 2^-17 of itself beside its share.

Nothing averages the errors of so few weights out; sums are within 2^-18 (test_gpu_sample.py), so the prefix's end is
certain.  The noise favours the token after the prefix, or its last one."""
import numpy as np
import pytest
import torch

from test_gpu_sample import check, gumbel

pytestmark = pytest.mark.gpu
F = np.float32


def rows(m, vocab, heavy, seed, rest):
    """Logits with `heavy` tokens within 4 of the largest and the others `rest` below, temperatures, and the share of
    the first 1 .. heavy of them (64-bit, of the weights of fp32 z)."""
    rng = np.random.default_rng(seed)
    x = (rng.normal(size=(m, vocab)) + rest).astype(F)
    t = rng.uniform(0.5, 1.5, m).astype(F)
    at = np.stack([rng.permutation(vocab)[:heavy] for _ in range(m)])
    np.put_along_axis(x, at, np.sort(rng.uniform(0, 4, (m, heavy)), 1)[:, ::-1].astype(F), 1)
    z = ((x - x.max(1, keepdims=True)).astype(F) * (F(1) / t)[:, None]).astype(F)
    w = np.exp(z.astype(np.float64))
    mass = np.cumsum(np.take_along_axis(w, at, 1), 1) / w.sum(1, keepdims=True)
    return torch.from_numpy(x), t, at, mass


@pytest.mark.parametrize("m,vocab,some", [(300, 4000, None), (320, 131072, 40), (3, 100003, None)])
@pytest.mark.parametrize("heavy,rest", [(2, -60), (3, -60), (2, -14), (4, -14)])
@pytest.mark.parametrize("side", ["below", "above"])
def test_share_of_heavy_tokens(m, vocab, some, heavy, rest, side):
    x, t, at, mass = rows(m, vocab, heavy, heavy + m, rest)
    last = np.arange(m) % (heavy - 1) if heavy > 2 else np.zeros(m, int)  # the prefix's last token, counted from 0
    r = np.arange(m)
    p = (mass[r, last] * (1 + (-2.0 ** -17 if side == "below" else 2.0 ** -17))).astype(F)
    g = gumbel(m, vocab, 1)
    g[r, at[r, last + 1]] += 100  # kept only if the prefix goes on
    check(x, g, t=t, p=p, rows=None if some is None else range(0, m, m // some))
    g[r, at[r, last + 1]] -= 100
    g[r, at[r, last]] += 100
    check(x, g, t=t, p=p, rows=None if some is None else range(0, m, m // some))
