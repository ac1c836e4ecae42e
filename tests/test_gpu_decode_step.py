"""The decode-step example against a plain forward pass in 64 bits without a cache, and its CUDA graph against eager steps.

The plain form runs every sequence whole, with W_eff = W_base + alpha * sign of its variant, all
positions at once under a causal mask.  Bound of the logits: a layer rounds to bf16 at most 20
times between two points of the residual stream (the weights of its 7 linears, their 7 outputs, 2
norms, rotation, attention, the product of gate and up, the stream itself), each by at most 2^-8 of its value; norms and
the linears pass relative errors of whole rows on as they are, and scores are too small
(below 1) for the softmax to raise them.  Added up linearly, relative to the row's norm: layers * 20 * 2^-8.  An 8-bit cache adds up to
2^-4 of K and V per layer."""
import numpy as np
import pytest
import torch

import step_ref as ref
from bit_delta_tenant_gb300 import bitdelta as bd
from bit_delta_tenant_gb300 import synth
from bit_delta_tenant_gb300.decode_step import Shape, Tenants

pytestmark = pytest.mark.gpu

SHAPE = Shape(layers=2, hidden=256, q_heads=4, kv_heads=2, head_dim=64, mlp=512, vocab=1001)
VARIANTS = [2, 0, 1, 2, 0]
PROMPTS = [1, 2, 23, 17, 9]
STEPS = 10
SETTINGS = dict(temperature=[0.0, 0.8, 1.0, 0.7, 1.3], top_k=[0, 20, 0, 0, 40], top_p=[1.0, 1.0, 0.9, 1.0, 0.8],
                min_p=[0.0, 0.0, 0.0, 0.05, 0.01])


def start(kv8):
    t = Tenants(SHAPE, 3, VARIANTS, max(PROMPTS) + STEPS, page_size=16, kv_e4m3=kv8, seed=3)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(0, SHAPE.vocab, (n,), generator=g).tolist() for n in PROMPTS]
    for i, p in enumerate(prompts):
        t.prefill(i, p, piece=5)
    t.sampling(**SETTINGS)
    return t, prompts


def run(t, step):
    g = synth.generator(5, "cuda")
    seen = []
    for _ in range(STEPS):
        t.draw_noise(g)
        step()
        seen.append([x.clone().cpu() for x in (t.logits, t.noise, t.tokens, t.logprob)])
    assert bd.bd_get_device_status() == bd.BD_OK
    return seen


def effective(w, v):
    bits = np.unpackbits(w.bits[v].cpu().numpy(), axis=1, bitorder="little").astype(np.float64)
    return ref.f64(w.base) + float(w.alpha[v].item()) * (2 * bits - 1)


def plain_logits(t, v, tokens):
    s, n = t.shape, len(tokens)
    norms, h = ref.f64(t.norms)[:, v], ref.f64(t.embedding)[tokens]
    rope = ref.f64(t.rope)[:n]

    def norm(i, x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + s.eps) * norms[i]

    for i, layer in enumerate(t.layers):
        w = {name: effective(m, v) for name, m in layer.items()}
        y = norm(2 * i, h)
        q, k, val = ((y @ w[name].T).reshape(n, -1, s.head_dim) for name in "qkv")
        q, k = ref.rotated(q, rope), ref.rotated(k, rope)
        out = np.stack([ref.attention(q[j], k[:j + 1], val[:j + 1], s.head_dim ** -0.5)[0] for j in range(n)])
        h = h + out.reshape(n, -1) @ w["o"].T
        y = norm(2 * i + 1, h)
        gate = y @ w["gate"].T
        h = h + (gate / (1 + np.exp(-gate)) * (y @ w["up"].T)) @ w["down"].T
    return norm(2 * s.layers, h) @ effective(t.head, v).T


@pytest.mark.parametrize("kv8", [False, True])
def test_generation_matches_a_plain_forward_pass(kv8):
    t, prompts = start(kv8)
    seen = run(t, t.step)
    bound = SHAPE.layers * (20 * 2.0 ** -8 + (2.0 ** -4 if kv8 else 0))
    for i, v in enumerate(VARIANTS):
        new = [int(s[2][i]) for s in seen]
        plain = plain_logits(t, v, prompts[i] + new[:-1])[len(prompts[i]) - 1:]
        got = np.stack([ref.f64(s[0][i]) for s in seen])
        off = np.linalg.norm(got - plain, axis=1) / np.linalg.norm(plain, axis=1)
        assert off.max() <= bound, (i, off)
        for s in seen:  # the draw, from the logits that it was made from
            want, logprob = ref.sample(s[0][i].float().numpy(), s[1][i].numpy(), SETTINGS["temperature"][i], SETTINGS["top_k"][i],
                                       SETTINGS["top_p"][i], SETTINGS["min_p"][i])
            assert int(s[2][i]) == want
            assert abs(float(s[3][i]) - logprob) <= 1e-3


def test_graph_gives_what_eager_steps_give():
    t, _ = start(False)
    eager = run(t, t.step)
    t, _ = start(False)
    t.draw_noise(synth.generator(6, "cuda"))
    graph = t.capture()
    replayed = run(t, graph.replay)
    for a, b in zip(eager, replayed):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
