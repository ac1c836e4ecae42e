"""bd_rmsnorm on the GPU against its definition in 64 bits.

Bounds.  The sum of n squares is added in at most 32 + 5 + 32 steps, so rsqrt(mean) is within
2^-18 of its value, and y within 2^-17 before its rounding; bf16 rounds to 2^-8 of the value, e4m3 to
2^-4 of it or half of its smallest step, 2^-10 scales."""
import numpy as np
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd
from step_ref import f64, randn

pytestmark = pytest.mark.gpu
EPS = 1e-5


def reference(x, residual, weight, ids):
    h = f64(x) + (0 if residual is None else f64(residual))
    w = f64(weight).reshape(-1, x.shape[1])
    w = w[0] if ids is None else w[ids.numpy()]
    with np.errstate(all="ignore"):
        return h, h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * w


def make(m, n, variants, residual, seed=0):
    x = randn((m, n), seed).bfloat16()
    r = randn((m, n), seed + 1, 3.0).bfloat16() if residual else None
    w = (1 + randn((variants, n), seed + 2, 0.2)).bfloat16()
    ids = torch.from_numpy(np.random.default_rng(seed).integers(0, variants, m).astype(np.int32)) if variants > 1 else None
    return x, r, w, ids


def cuda(t):
    return None if t is None else t.cuda()


def check_bf16(got, ref):
    assert np.all(np.abs(f64(got) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -15) + 1e-30)


@pytest.mark.parametrize("m", [1, 3, 64])
@pytest.mark.parametrize("n", [8, 16, 1016, 1024, 1032, 2048, 4096, 5120, 8192, 8200, 16384, 20000, 32768])
def test_bf16(m, n):
    x, r, w, ids = make(m, n, 1 + m % 3, residual=n % 16 == 0, seed=m + n)
    y, ro = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y, residual=cuda(r), residual_out=ro, weight_ids=cuda(ids))
    h, ref = reference(x, r, w, ids)
    check_bf16(y, ref)
    assert np.all(np.abs(f64(ro) - h) <= np.abs(h) * (2.0 ** -8 + 2.0 ** -20))
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("m,n,per_row", [(1, 128, False), (5, 1152, False), (64, 8192, False), (2, 32768, False),
                                         (1, 8, True), (7, 1000, True), (64, 8192, True), (3, 20000, True)])
def test_8_bits(m, n, per_row):
    x, r, w, ids = make(m, n, 3, residual=True, seed=n)
    x[0, : n // 2] = 0
    r[0, : n // 2] = 0  # with 128 columns a scale, some groups are all zero
    y = torch.empty((m, n), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((m, 1 if per_row else n // 128), dtype=torch.float32, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y, residual=r.cuda(), y_scale=s, weight_ids=cuda(ids))
    _, ref = reference(x, r, w, ids)
    ref = ref.reshape(*s.shape, -1)
    top = np.abs(ref).max(-1)
    scale = f64(s)
    assert np.all(scale[top == 0] == 1)
    assert np.all(np.abs(scale - top / 448)[top > 0] <= (top / 448 * 2.0 ** -16)[top > 0])
    got = f64(y.float()).reshape(ref.shape) * scale[..., None]
    assert np.all(np.abs(got - ref) <= np.abs(ref) * (2.0 ** -4 + 2.0 ** -10) + scale[..., None] * 2.0 ** -9.9 * (ref != 0))


@pytest.mark.parametrize("top", [1e-45, 1e-40, 1e-38, 1e-35, 1e-30, 1e-10, 1e10])
def test_8_bits_of_tiny_and_large_rows(top):
    """No scale overflows its reciprocal: what is too small for a scale becomes zero, nothing becomes NaN."""
    x = (torch.arange(256).view(2, 128).float() / 256 * top).bfloat16()
    y = torch.empty((2, 128), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((2, 1), dtype=torch.float32, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w, EPS, y, y_scale=s)
    _, ref = reference(x, None, torch.ones((1, 128)).bfloat16(), None)
    got = f64(y.float()) * f64(s)
    tiny = np.abs(f64(x)).max(1) < 2.0 ** -100
    assert np.all(f64(s)[tiny] == 1) and np.all(got[tiny] == 0)
    tol = np.abs(ref) * (2.0 ** -4 + 2.0 ** -10) + f64(s) * 2.0 ** -9.9
    assert np.all(np.abs(got - ref)[~tiny] <= tol[~tiny])


def test_residual_in_place_and_no_residual_output():
    x, r, w, _ = make(9, 4096, 1, True)
    rd, y, y2 = r.cuda(), torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w[0].cuda(), EPS, y2, residual=rd)
    assert torch.equal(rd.cpu(), r)
    bd.bd_rmsnorm(x.cuda(), w[0].cuda(), EPS, y, residual=rd, residual_out=rd)
    h, ref = reference(x, r, w, None)
    check_bf16(y, ref)
    assert torch.equal(y, y2)
    assert np.all(np.abs(f64(rd) - h) <= np.abs(h) * (2.0 ** -8 + 2.0 ** -20))


def test_zero_rows_nan_rows_and_large_values_stay_in_their_row():
    x, _, w, _ = make(5, 512, 1, False)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    x[4] = 1e18  # its squares stay in fp32, 512e36
    y = torch.empty_like(x, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y)
    _, ref = reference(x, None, w, None)
    check_bf16(y[[0, 1, 4]], ref[[0, 1, 4]])
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 9]) and (y[3, :9] == 0).all()


def test_bad_weight_id_flags_and_leaves_the_row():
    x, _, w, _ = make(4, 256, 2, False)
    ids = torch.tensor([0, 2, 1, -1], dtype=torch.int32).cuda()
    y = torch.full_like(x, 7.0, device="cuda")
    bd.bd_rmsnorm(x.cuda(), w.cuda(), EPS, y, weight_ids=ids)
    assert bd.bd_get_device_status() == bd.BD_ERR_BAD_VARIANT_ID
    assert (y[[1, 3]] == 7).all() and not (y[[0, 2]] == 7).all()
    assert bd.bd_get_device_status() == bd.BD_OK


def test_empty_batch_and_refusals():
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    bd.bd_rmsnorm(e, torch.ones(256, dtype=torch.bfloat16, device="cuda"), EPS, e.clone())
    x = torch.ones((2, 256), dtype=torch.bfloat16, device="cuda")
    w = x[0].clone()
    for bad in (dict(y=x.float()), dict(y=x.t().contiguous().t()), dict(residual=x[:1]), dict(weight_ids=torch.zeros(2).cuda()),
                dict(y_scale=torch.ones((2, 3), device="cuda")), dict(weight=w[:128])):
        a = dict(weight=w, y=torch.empty_like(x))
        a.update(bad)
        with pytest.raises(ValueError):
            bd.bd_rmsnorm(x, a.pop("weight"), EPS, a.pop("y"), **a)
    with pytest.raises(bd.BitDeltaError) as e:
        bd.bd_rmsnorm(x, w, -1.0, torch.empty_like(x))
    assert e.value.status == bd.BD_ERR_INVALID_ARG
