"""bd_rmsnorm at the ends of fp32's range: squares beyond it under a mean within it, and rows next to zero without eps.

Bounds as in test_gpu_step_norm.py; rsqrt(mean) is within one rounding more where each square is divided by n by itself."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import f64, randn
from test_gpu_step_norm import EPS, check_bf16, make, reference

pytestmark = pytest.mark.gpu


def outliers(n, at):
    """Rows with an element whose square alone passes fp32, several in one 16-byte piece, and one of each sign far apart."""
    x, _, w, _ = make(4, n, 1, False, seed=n)
    x[0, at] = 2e19
    first = at // 8 * 8
    x[1, first:first + 8] = 1.9e19 / 8 ** 0.5 * (n / 512) ** 0.5  # none passes it, their sum does
    x[2, 0], x[2, n - 1] = 2.5e19, -1.9e19
    return x, w


@pytest.mark.parametrize("n,at", [(1024, 0), (1024, 1023), (4096, 77), (8192, 8191), (20000, 12345), (32768, 32767), (32768, 5)])
def test_squares_beyond_the_range(n, at):
    x, w = outliers(n, at)
    y = torch.empty_like(x, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y)
    _, ref = reference(x, None, w, None)
    check_bf16(y, ref)
    assert np.abs(f64(y)[0, at]) > 1


@pytest.mark.parametrize("n,per_row", [(1024, False), (8192, False), (32768, False), (20000, True)])
def test_squares_beyond_the_range_8_bits(n, per_row):
    x, w = outliers(n, n // 3)
    y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((4, 1 if per_row else n // 128), dtype=torch.float32, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y, y_scale=s)
    _, ref = reference(x, None, w, None)
    ref = ref.reshape(*s.shape, -1)
    top, scale = np.abs(ref).max(-1), f64(s)
    assert np.all(np.abs(scale - top / 448) <= top / 448 * 2.0 ** -16)
    got = f64(y.float()).reshape(ref.shape) * scale[..., None]
    assert np.all(np.abs(got - ref) <= np.abs(ref) * (2.0 ** -4 + 2.0 ** -10) + scale[..., None] * 2.0 ** -9.9)


@pytest.mark.parametrize("n", [512, 8192, 32768])
def test_small_rows_without_eps(n):
    """Squares of about 2^-120: their sum keeps its digits."""
    x = (randn((3, n), n) * 2.0 ** -60).bfloat16()
    w = torch.ones((1, n), dtype=torch.bfloat16)
    y = torch.empty_like(x, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), 0.0, y)
    h = f64(x)
    check_bf16(y, h / np.sqrt((h * h).mean(1, keepdims=True)))


def test_infinities_and_nan_stay_in_their_row():
    x = randn((4, 2048), 3).bfloat16()
    x[1, 5], x[2, 9] = float("inf"), float("nan")
    w = torch.ones((1, 2048), dtype=torch.bfloat16)
    y = torch.empty_like(x, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y)
    _, ref = reference(x[[0, 3]], None, w, None)
    check_bf16(y[[0, 3]], ref)
    assert torch.isnan(y[2]).all() and torch.isnan(y[1, 5])
