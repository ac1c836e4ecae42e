"""The generation example where its score cap, its scaled positions and its attention decide the logits, against a plain forward pass in 64 bits.

Weights are the example's with q, k, v and o times 6 and the embedding a quarter: scores spread by some 3.8 about a cap of 3, and attention outweighs what it
is added to.  The plain pass without the cap, without the scaling or without attention lies outside the bound, which is asserted beside it.

Bound.  A layer rounds to bf16 20 times between two points of the stream (see test_gpu_decode_step), each by up to 2^-8 of a value, 2^-8 / sqrt(3) in
the mean square, independently: sqrt(20) of that, 0.0101.  A score of spread 3.8 is made of q and k, each after 4 such roundings: off by
sqrt(2) sqrt(4) 3.8 2^-8 / sqrt(3) = 0.0242 in the mean square (the cap lets less through), and so are the weights relative to each other and the rows that they
make.  Together 0.0262 a layer, 0.0524 for two one after the other; rows are held to four times that, 0.21.

Over a 4-bit cache a rounding may tip a value into the next code, so the plain pass attends to what the cache holds, and K and V of its own are compared
with that: half a unit of 6 at most beside each other's rounding, a quarter of the row's norm as in test_gpu_decode_step_long, and the 0.21 of the rows
that they are made from."""
import numpy as np
import pytest
import torch

import step_ref as ref
import test_gpu_decode_step as base
from bit_delta_tenant_gb300 import bitdelta as bd
from bit_delta_tenant_gb300 import synth
from bit_delta_tenant_gb300.decode_step import Shape, Tenants

pytestmark = pytest.mark.gpu

SHAPE = Shape(layers=2, hidden=256, q_heads=4, kv_heads=2, head_dim=64, mlp=512, vocab=1001, rope_base=1e4, rope_factor=32.0, rope_original=16,
              score_cap=3.0)
VARIANTS, PROMPTS, STEPS, BOUND = [2, 0, 1], [30, 75, 2], 6, 0.21


def plain(t, v, tokens, cached=None, cap=True, scaling=True, attend=True):
    """Logits of every token, and each layer's K and V; `cached` K and V are attended to instead."""
    s, n = t.shape, len(tokens)
    norms, h = ref.f64(t.norms)[:, v], ref.f64(t.embedding)[tokens]
    f = s.rope_base ** (-2.0 * np.arange(s.head_dim // 2) / s.head_dim)
    if scaling:
        keep = np.clip((s.rope_original * f / (2 * np.pi) - 1) / 3, 0, 1)
        f = f * (keep + (1 - keep) / s.rope_factor)
    a = np.arange(n)[:, None] * f
    rope = np.concatenate([np.cos(a), np.sin(a)], 1)

    def norm(i, x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + s.eps) * norms[i]

    made = []
    for i, layer in enumerate(t.layers):
        w = {name: base.effective(m, v) for name, m in layer.items()}
        y = norm(2 * i, h)
        q, k, val = ((y @ w[name].T).reshape(n, -1, s.head_dim) for name in "qkv")
        q, k = ref.rotated(q, rope), ref.rotated(k, rope)
        made.append((k, val))
        if cached is not None:
            k, val = cached[i]
        x = np.einsum("ihgd,jhd->hgij", q.reshape(n, s.kv_heads, -1, s.head_dim), k) * s.head_dim ** -0.5
        x = s.score_cap * np.tanh(x / s.score_cap) if cap else x
        x = np.where(np.tril(np.ones((n, n), bool)), x, -np.inf)
        x = np.exp(x - x.max(-1, keepdims=True))
        out = np.einsum("hgij,jhd->ihgd", x / x.sum(-1, keepdims=True), val).reshape(n, -1)
        h = h + (out if attend else 0 * out) @ w["o"].T
        y = norm(2 * i + 1, h)
        gate = y @ w["gate"].T
        h = h + (gate / (1 + np.exp(-gate)) * (y @ w["up"].T)) @ w["down"].T
    return norm(2 * s.layers, h) @ base.effective(t.head, v).T, made


def tenants(**kw):
    t = Tenants(SHAPE, 3, VARIANTS, max(PROMPTS) + STEPS, page_size=16, seed=3, **kw)
    for layer in t.layers:
        for name in ("q", "k", "v", "o"):
            layer[name].base.mul_(6)
    t.embedding.mul_(0.25)
    t.draw_noise(synth.generator(5, "cuda"))
    return t


def apart(x, y):
    return np.linalg.norm(x - y, axis=-1) / np.linalg.norm(y, axis=-1)


def cached_rows(t, i, n):
    out = []
    for cache in t.caches:
        k, v = (torch.empty((n, SHAPE.kv_heads, SHAPE.head_dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        bd.bd_kv_read(cache, t.page_table[i:i + 1], torch.tensor([0, n], dtype=torch.int32, device="cuda"), k, v)
        out.append((ref.f64(k), ref.f64(v)))
    return out


@pytest.mark.parametrize("kv4", [False, True])
def test_the_rules_decide_the_logits(kv4):
    t = tenants(kv_e2m1=kv4)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(0, SHAPE.vocab, (n,), generator=g).tolist() for n in PROMPTS]
    for i, p in enumerate(prompts):
        t.prefill(i, p, piece=16)
    noise = synth.generator(5, "cuda")
    drawn, logits = [], []
    for _ in range(STEPS):
        t.draw_noise(noise)
        t.step()
        drawn.append(t.tokens.tolist()), logits.append(ref.f64(t.logits))
    for i, v in enumerate(VARIANTS):
        tokens = prompts[i] + [d[i] for d in drawn[:-1]]
        last = slice(len(prompts[i]) - 1, None)
        cached = cached_rows(t, i, len(tokens)) if kv4 else None
        want, made = plain(t, v, tokens, cached)
        got = np.stack([x[i] for x in logits])
        off = apart(got, want[last])
        assert off.max() <= BOUND, (i, off)
        if kv4:
            for own, held in zip(made, cached):
                for x, y in zip(own, held):
                    assert apart(y.reshape(len(tokens), -1), x.reshape(len(tokens), -1)).max() <= 0.25 + BOUND
        if len(prompts[i]) > 20:  # over few tokens each of them changes little
            for other in (dict(cap=False), dict(scaling=False), dict(attend=False)):
                assert apart(plain(t, v, tokens, **other)[0][last], plain(t, v, tokens)[0][last]).min() > 1.5 * BOUND, (i, other)
    assert bd.bd_get_device_status() == bd.BD_OK


def test_prompts_in_pieces_and_token_by_token():
    """The same sequence prefilled at once, in pieces, and fed token by token to the step: within twice the bound of one against the plain pass."""
    tokens = list(range(7, 47))
    seen = []
    for piece in (64, 16, 1):
        t = tenants()
        t.prefill(1, tokens, piece=piece)
        t.step()
        seen.append(ref.f64(t.logits[1]))
    t = tenants()
    t.prefill(1, tokens[:1])
    for token in tokens:
        t.tokens[1] = token
        t.step()
    seen.append(ref.f64(t.logits[1]))
    for x in seen[1:]:
        assert apart(x, seen[0]) <= 2 * BOUND
