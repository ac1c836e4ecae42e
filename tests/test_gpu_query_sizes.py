"""Queries next to either end of bf16's range, over caches whose products take them times a power of two: scores are as they
would be for ordinary queries, as `scale` takes them back there.

Bounds are test_gpu_prompt's and test_gpu_four_bits's for ordinary queries: powers of two change no bit."""
import pytest
import torch

import test_gpu_four_bits as four
import test_gpu_prompt as prompt
from bit_delta_tenant_gb300 import bitdelta as bd
from long_ref import Pool
from step_ref import randn

pytestmark = pytest.mark.gpu
POWERS = [-103, 100, 101, 110, 118]
# as bf16 numbers such queries make products next to fp32's subnormals
SCALED = [(kv, p) for kv in prompt.KINDS for p in POWERS]


def queries(n, heads, dim, power):
    """One head much smaller than the others, one of zeros."""
    q = randn((n, heads, dim), 9, 1.0)
    q[:, 1] *= 0.03125
    q[:, 2] = 0.0
    return (q * 2.0 ** power).bfloat16()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv,power", SCALED + [("e2m1", -116)])
def test_prompts(kv, dim, power):
    new, past = [20, 3], [0, 200]
    pool = Pool([20, 203], 2, dim, 16, kv, seed=1)
    q = queries(23, 8, dim, power)
    rule = dict(scale=dim ** -0.5 * 2.0 ** -power)
    out, lse = prompt.run(pool, q, new, **rule)
    prompt.check(pool, q, new, out, lse, **rule)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 8), (128, 32)])
@pytest.mark.parametrize("kv,power", SCALED + [("e2m1", -116), ("e4m3", -116)])
def test_single_tokens(kv, dim, heads, power):
    pool = Pool([700, 3, 129], 2, dim, 16, kv, seed=2)
    q = queries(3, heads, dim, power)
    rule = dict(scale=dim ** -0.5 * 2.0 ** -power)
    out, lse = four.decode(pool, q, **rule)
    four.check(pool, q, out, lse, **rule)
    assert bd.bd_get_device_status() == bd.BD_OK


@pytest.mark.parametrize("kv", prompt.KINDS)
def test_the_largest_and_smallest_numbers(kv):
    """Heads of bf16's largest value, or of nothing but its subnormals, with a scale that makes ordinary scores of one of them."""
    pool = Pool([40, 40], 1, 64, 16, kv, seed=3, k_std=0.0625)
    q = torch.zeros((2, 2, 64))
    q[:, 0, ::7] = torch.finfo(torch.bfloat16).max
    q[:, 1, ::7] = 2.0 ** -133
    q = q.bfloat16()
    rule = dict(scale=2.0 ** -126)  # the second head's scores are 0
    out, lse = four.decode(pool, q, **rule)
    four.check(pool, q, out, lse, **rule)
    out, lse = prompt.run(pool, q, [1, 1], **rule)
    prompt.check(pool, q, [1, 1], out, lse, **rule)
