"""The generation example with a 4-bit cache, scaled positions and capped scores against a plain forward pass in 64 bits.

Bound as in test_gpu_decode_step: 20 roundings of 2^-8 per layer, and for the cache the error of a 4-bit value.  A group's
values are within a quarter of a unit to one unit of 6 units, at least a sixth of the value or 1/24 of the group's largest, and the scale's rounding
is a sixteenth: K and V are off by less than a quarter of their rows' norms, once per layer."""
import numpy as np
import pytest
import torch

import step_ref as ref
import test_gpu_decode_step as base
from bit_delta_tenant_gb300 import bitdelta as bd
from bit_delta_tenant_gb300.decode_step import Shape, Tenants

pytestmark = pytest.mark.gpu

SHAPE = Shape(layers=2, hidden=256, q_heads=4, kv_heads=2, head_dim=64, mlp=512, vocab=1001, rope_base=1e4, rope_factor=8.0, rope_original=64,
              score_cap=3.0)


def plain_logits(t, v, tokens, cap):
    s, n = t.shape, len(tokens)
    norms, h = ref.f64(t.norms)[:, v], ref.f64(t.embedding)[tokens]
    i = np.arange(s.head_dim // 2)
    f = s.rope_base ** (-2.0 * i / s.head_dim)
    keep = np.clip((s.rope_original * f / (2 * np.pi) - 1) / 3, 0, 1)
    a = np.arange(n)[:, None] * (f * (keep + (1 - keep) / s.rope_factor))
    rope = np.concatenate([np.cos(a), np.sin(a)], 1)

    def norm(i, x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + s.eps) * norms[i]

    for i, layer in enumerate(t.layers):
        w = {name: base.effective(m, v) for name, m in layer.items()}
        y = norm(2 * i, h)
        q, k, val = ((y @ w[name].T).reshape(n, -1, s.head_dim) for name in "qkv")
        q, k = ref.rotated(q, rope), ref.rotated(k, rope)
        g = s.q_heads // s.kv_heads
        x = np.einsum("ihgd,jhd->hgij", q.reshape(n, s.kv_heads, g, -1), k) * s.head_dim ** -0.5
        x = np.where(np.tril(np.ones((n, n), bool)), cap * np.tanh(x / cap), -np.inf)
        x = np.exp(x - x.max(-1, keepdims=True))
        out = np.einsum("hgij,jhd->ihgd", x / x.sum(-1, keepdims=True), val)
        h = h + out.reshape(n, -1) @ w["o"].T
        y = norm(2 * i + 1, h)
        gate = y @ w["gate"].T
        h = h + (gate / (1 + np.exp(-gate)) * (y @ w["up"].T)) @ w["down"].T
    return norm(2 * s.layers, h) @ base.effective(t.head, v).T


@pytest.mark.parametrize("kv4", [False, True])
def test_generation_matches_a_plain_forward_pass(kv4):
    t = Tenants(SHAPE, 3, base.VARIANTS, max(base.PROMPTS) + base.STEPS, page_size=16, seed=3, kv_e2m1=kv4)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(0, SHAPE.vocab, (n,), generator=g).tolist() for n in base.PROMPTS]
    for i, p in enumerate(prompts):
        t.prefill(i, p, piece=9)
    t.sampling(**base.SETTINGS)
    seen = base.run(t, t.step)
    bound = SHAPE.layers * (20 * 2.0 ** -8 + (0.25 if kv4 else 0))
    for i, v in enumerate(base.VARIANTS):
        new = [int(s[2][i]) for s in seen]
        plain = plain_logits(t, v, prompts[i] + new[:-1], SHAPE.score_cap)[len(prompts[i]) - 1:]
        got = np.stack([ref.f64(s[0][i]) for s in seen])
        off = np.linalg.norm(got - plain, axis=1) / np.linalg.norm(plain, axis=1)
        assert off.max() <= bound, (i, off)
    assert bd.bd_get_device_status() == bd.BD_OK


def test_the_same_tokens_from_a_graph():
    def tenants():
        t = Tenants(SHAPE, 3, base.VARIANTS, max(base.PROMPTS) + base.STEPS, page_size=16, seed=3, kv_e2m1=True)
        for i, n in enumerate(base.PROMPTS):
            t.prefill(i, list(range(n)), piece=100)
        t.sampling(**base.SETTINGS)
        return t

    t = tenants()
    eager = base.run(t, t.step)
    t = tenants()
    t.draw_noise(torch.Generator(device="cuda").manual_seed(6))
    graph = t.capture()
    for a, b in zip(eager, base.run(t, graph.replay)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
