"""bd_sample where most of a row is masked by large negative numbers instead of -inf, as constrained decoding does.

Masked tokens stand before, between and after live ones in the logits that one thread sums, and fill whole
slices.  Bounds as in test_gpu_sample.py; a masked token weighs nothing."""
import numpy as np
import pytest
import torch

from test_gpu_sample import DTYPES, check, gumbel, logits

pytestmark = pytest.mark.gpu

KINDS = {"unfiltered": {}, "top-p": dict(p=0.9), "top-k": dict(k=50), "top-k and top-p": dict(k=3000, p=0.8), "min-p": dict(low=0.05),
         "greedy": dict(t=0.0)}


def masked(m, vocab, dtype, mask):
    """Rows with a masked beginning, a random 95 % masked, every second 16 bytes masked, and a masked end."""
    x = logits(m, vocab, vocab, dtype)
    rng = np.random.default_rng(vocab)
    low = torch.finfo(dtype).min if mask == "lowest" else float(mask)
    at = torch.arange(vocab)
    for r in range(m):
        kind = r % 5
        if kind == 0:
            hide = at < vocab * 0.95
        elif kind == 1:
            hide = torch.from_numpy(rng.random(vocab) < 0.95)
        elif kind == 2:
            hide = at // 8 % 2 == 0
        elif kind == 3:
            hide = at > vocab // 20
        else:
            hide = (at < vocab - 3) & (at != vocab // 2)
        x[r, hide] = low
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mask", ["lowest", "-1e30", "-1e10"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [0.6, 1.0, 1.3])
def test_large_negative_masks(dtype, mask, kind, t):
    """A cluster per row, with four to eight units to a thread."""
    m, vocab = 5, 128256
    check(masked(m, vocab, dtype, mask), gumbel(m, vocab, 3), **{"t": t, **KINDS[kind]})


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_large_negative_masks_one_cta_per_row(dtype, kind):
    m, vocab = 320, 20003
    check(masked(m, vocab, dtype, "lowest"), gumbel(m, vocab, 4), rows=[0, 1, 2, 3, 4, 317, 318, 319], **KINDS[kind])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_masks_of_several_values(dtype, kind):
    """One masked value raised by another before the first live token comes."""
    m, vocab = 2, 60000
    x = logits(m, vocab, 5, dtype)
    x[:, :20000], x[:, 20000:40000], x[0, 40000:55000] = torch.finfo(dtype).min, -1e30, -3e5
    check(x, gumbel(m, vocab, 5), **KINDS[kind])
