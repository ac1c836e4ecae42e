"""Text generation for many tenants over one base model: prompts, then one token per sequence and step.

Every sequence names its variant.  A layer of a step is

    norm -> q, k, v -> rotary positions and cache write -> attention over the cache -> o
    -> residual addition and norm -> gate, up -> silu(gate) * up -> down

with all linears multi-tenant (bd_linear_grouped: shared base, per-variant packed delta) and the
norm weights chosen per token by variant (bd_rmsnorm); the last norm, the head and bd_sample end a step, each sequence with
its own sampling settings.  Nothing in a step depends on a host value, so a step is captured once
in a CUDA graph and replayed; positions advance on the device.

    python -m bit_delta_tenant_gb300.decode_step --layers 32 --sequences 64 --steps 64

Weights are random: the shapes are those of the Llama-3-8B-shape stack.  Prompts are processed
sequence by sequence in pieces; a piece attends to what is cached, itself included (bd_attention_prompt).  The cache holds
bf16, 8 or 4 bits; positions may be scaled for contexts beyond the model's own, scores capped.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from . import bitdelta as bd
from . import synth, workloads


@dataclass
class Shape:
    layers: int = 32
    hidden: int = 4096
    q_heads: int = 32
    kv_heads: int = 8
    head_dim: int = 128
    mlp: int = 14336
    vocab: int = 128256
    eps: float = 1e-5
    rope_base: float = 5e5
    rope_factor: float = 1.0    # by how much slow rotations are slowed down further, and the context
    rope_original: int = 8192   # that the others are told from them by
    score_cap: float = 0.0

    def matrices(self):
        """(name, n_out, n_in) of a layer's linears, as in workloads.LLAMA3_8B_STACK."""
        q, kv = self.q_heads * self.head_dim, self.kv_heads * self.head_dim
        return [("q", q, self.hidden), ("k", kv, self.hidden), ("v", kv, self.hidden), ("o", self.hidden, q),
                ("gate", self.mlp, self.hidden), ("up", self.mlp, self.hidden), ("down", self.hidden, self.mlp)]


def rope_table(positions: int, dim: int, base: float) -> torch.Tensor:
    """fp32 [positions, dim] on the CPU: cosines, then sines, of position * base^(-2i / dim), as bd_rotary_table makes them unscaled."""
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Matrix:
    """A base matrix and its variants' packed deltas."""

    def __init__(self, n_out, n_in, n_variants, g, sigma=0.02, alpha=1e-3):
        dev = g.device
        self.base = synth.bf16_normal((n_out, n_in), sigma, g, dev)
        self.bits = [torch.randint(0, 256, (n_out, n_in // 8), generator=g, device=dev, dtype=torch.uint8)
                     for _ in range(n_variants)]
        self.alpha = [torch.full((1,), alpha * (v + 1) / n_variants, device=dev) for v in range(n_variants)]


class Tenants:
    """The model, its variants, and the sequences being served with their cache."""

    def __init__(self, shape: Shape, n_variants: int, variants, max_tokens: int, page_size: int = 64,
                 kv_e4m3: bool = False, seed: int = 0, device="cuda", kv_e2m1: bool = False):
        self.shape, self.n_variants, self.max_tokens = shape, n_variants, max_tokens
        g = synth.generator(seed, device)
        m = self.m = len(variants)
        s, dev = shape, g.device
        self.variants = torch.tensor(variants, dtype=torch.int32, device=dev)
        self.embedding = synth.bf16_normal((s.vocab, s.hidden), 1.0, g, dev)
        self.layers = [{n: Matrix(o, i, n_variants, g) for n, o, i in s.matrices()} for _ in range(s.layers)]
        self.head = Matrix(s.vocab, s.hidden, n_variants, g)
        # norm weights of a layer's attention and MLP and of the head, per variant
        self.norms = (1 + 0.1 * torch.randn((2 * s.layers + 1, n_variants, s.hidden), generator=g, device=dev)).bfloat16()
        self.rope = torch.empty((max_tokens, s.head_dim), device=dev)
        bd.bd_rotary_table(self.rope, s.rope_base, factor=s.rope_factor, original=s.rope_original)
        pages = -(-max_tokens // page_size)
        order = torch.randperm(m * pages, generator=g, device=dev)  # a pool's free pages are in no order
        self.page_table = order.to(torch.int32).view(m, pages)
        pool = (m * pages, s.kv_heads, page_size, s.head_dim)
        kv, scales = (torch.float8_e4m3fn, pool[:3]) if kv_e4m3 else (torch.bfloat16, None)
        if kv_e2m1:  # two values to a byte, a scale byte for 16
            if kv_e4m3:
                raise ValueError("a cache holds 8 bits or 4")
            kv, scales, pool = torch.uint8, (*pool[:3], s.head_dim // 16), (*pool[:3], s.head_dim // 2)
        self.caches = [bd.KVCache(torch.empty(pool, dtype=kv, device=dev), torch.empty(pool, dtype=kv, device=dev),
                                  *([torch.empty(scales, dtype=torch.uint8, device=dev) for _ in range(2)] if scales else []))
                       for _ in range(s.layers)]
        self.attention_ws = torch.zeros((bd.bd_attention_workspace_size(self.caches[0], m, s.q_heads),), dtype=torch.uint8, device=dev)
        self.prompt_ws = torch.zeros((bd.bd_attention_prompt_workspace_size(self.caches[0], s.q_heads),), dtype=torch.uint8, device=dev)
        self.linear_ws = {}
        self.modes = [bd.BD_ALPHA_SCALAR] * n_variants
        self.tokens = torch.zeros((m,), dtype=torch.int32, device=dev)     # each sequence's last token, not cached yet
        self.positions = torch.zeros((m,), dtype=torch.int32, device=dev)  # and its position
        self.logits = torch.empty((m, s.vocab), dtype=torch.bfloat16, device=dev)
        self.noise = torch.empty((m, s.vocab), dtype=torch.float32, device=dev)
        self.logprob = torch.empty((m,), dtype=torch.float32, device=dev)
        self.settings = {}

    def sampling(self, temperature=None, top_k=None, top_p=None, min_p=None):
        """Settings per sequence (lists, or None to leave a filter off)."""
        kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
        given = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        self.settings = {n: torch.tensor(v, dtype=kinds[n], device=self.tokens.device) for n, v in given.items() if v is not None}

    def _linear(self, w: Matrix, x, ids, y=None):
        m, (n_out, n_in) = x.shape[0], w.base.shape
        key = (m, n_out, n_in)
        if key not in self.linear_ws:
            size = bd.bd_linear_grouped_workspace_size(m, self.n_variants, n_out, n_in)
            self.linear_ws[key] = torch.empty((size,), dtype=torch.uint8, device=x.device)
        y = torch.empty((m, n_out), dtype=torch.bfloat16, device=x.device) if y is None else y
        bd.bd_linear_grouped(x, ids, w.base, w.bits, w.alpha, self.modes, y, self.linear_ws[key])
        return y

    def _norm(self, i, x, ids, residual=None):
        """Norm i of x, or of residual + x, which replaces the residual."""
        y = torch.empty_like(x)
        bd.bd_rmsnorm(x, self.norms[i], self.shape.eps, y, residual=residual, residual_out=residual, weight_ids=ids)
        return y

    def _layers(self, tokens, ids, positions, attend, seq_ids=None, table=None):
        """The residual stream's last addend and the stream before it, of one token per row."""
        s = self.shape
        h = self.embedding[tokens]
        x, n = None, tokens.shape[0]
        for i, w in enumerate(self.layers):
            y = self._norm(2 * i, h, ids) if x is None else self._norm(2 * i, x, ids, h)
            q, k, v = (self._linear(w[name], y, ids).view(n, -1, s.head_dim) for name in "qkv")
            bd.bd_kv_append(self.caches[i], q, k, v, positions, self.page_table if table is None else table, self.rope, q,
                            seq_ids=seq_ids)
            x = self._linear(w["o"], attend(self.caches[i], q).view(n, -1), ids)
            y = self._norm(2 * i + 1, x, ids, h)
            gate, up = self._linear(w["gate"], y, ids), self._linear(w["up"], y, ids)
            x = self._linear(w["down"], (torch.nn.functional.silu(gate.float()) * up).bfloat16(), ids)
        return x, h

    def prefill(self, i: int, prompt, piece: int = 512) -> None:
        """Cache all of a prompt of sequence i but its last token, which the next step takes."""
        s, dev = self.shape, self.tokens.device
        prompt = torch.as_tensor(prompt)
        if not 0 <= i < self.m:
            raise ValueError(f"a sequence is one of 0 to {self.m - 1}")
        if prompt.dim() != 1 or not 0 < prompt.numel() <= self.max_tokens:
            raise ValueError(f"a prompt has 1 to {self.max_tokens} tokens")
        if int(prompt.min()) < 0 or int(prompt.max()) >= s.vocab:  # rows of the embedding, unchecked from here on
            raise ValueError(f"a token is one of 0 to {s.vocab - 1}")
        prompt = prompt.to(dev, torch.int32)
        table = self.page_table[i:i + 1]

        for start in range(0, prompt.numel() - 1, piece):
            tokens = prompt[start:min(start + piece, prompt.numel() - 1)]
            n, end = tokens.numel(), start + tokens.numel()
            positions = torch.arange(start, end, dtype=torch.int32, device=dev)
            offsets = torch.tensor([0, n], dtype=torch.int32, device=dev)
            length = torch.tensor([end], dtype=torch.int32, device=dev)

            def attend(cache, q):
                out = torch.empty_like(q)
                bd.bd_attention_prompt(cache, q, offsets, table, length, out, self.prompt_ws, cap=s.score_cap)
                return out

            self._layers(tokens, self.variants[i:i + 1].repeat(n), positions, attend,
                         torch.zeros((n,), dtype=torch.int32, device=dev), table)
        self.tokens[i] = prompt[-1]
        self.positions[i] = prompt.numel() - 1

    def step(self) -> torch.Tensor:
        """One more token of every sequence; self.noise holds the Gumbel noise to draw with."""
        lengths = self.positions + 1

        def attend(cache, q):
            out = torch.empty_like(q)
            bd.bd_attention_decode(cache, q, self.page_table, lengths, out, self.attention_ws, cap=self.shape.score_cap)
            return out

        x, h = self._layers(self.tokens, self.variants, self.positions, attend)
        y = self._norm(2 * self.shape.layers, x, self.variants, h)
        self._linear(self.head, y, self.variants, self.logits)
        bd.bd_sample(self.logits, self.noise, self.tokens, logprob=self.logprob, **self.settings)
        self.positions += 1
        return self.tokens

    def draw_noise(self, g: torch.Generator) -> None:
        """Fresh Gumbel noise, -log of exponential draws."""
        self.noise.exponential_(generator=g).log_().neg_()

    def capture(self) -> torch.cuda.CUDAGraph:
        """One step as a CUDA graph.  (The step run before the capture leaves tokens, positions and cache as they were.)"""
        kept = self.tokens.clone(), self.positions.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()  # sizes workspaces; writes the cache at the position that the first replay writes again
        torch.cuda.current_stream().wait_stream(side)
        self.tokens.copy_(kept[0]), self.positions.copy_(kept[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=workloads.LLAMA3_8B_STACK["layers"])
    ap.add_argument("--sequences", type=int, default=64)
    ap.add_argument("--variants", type=int, default=14)
    ap.add_argument("--prompt", type=int, default=200, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--kv8", action="store_true", help="8-bit cache")
    ap.add_argument("--kv4", action="store_true", help="4-bit cache")
    ap.add_argument("--rope-factor", type=float, default=1.0, help="positions scaled for a context this many times the model's own")
    a = ap.parse_args()
    ids = synth.zipf_ids(a.sequences, a.variants, 1.1, 0).tolist()
    t = Tenants(Shape(layers=a.layers, rope_factor=a.rope_factor), a.variants, ids, a.prompt + a.steps, kv_e4m3=a.kv8, kv_e2m1=a.kv4)
    g = synth.generator(1, "cuda")
    for i in range(a.sequences):
        n = a.prompt - i * (a.prompt - 1) // a.sequences
        t.prefill(i, torch.randint(0, t.shape.vocab, (n,), generator=g, device="cuda"))
    # a quarter each: greedy, top-k, top-p, min-p
    kind = [i % 4 for i in range(a.sequences)]
    t.sampling(temperature=[0.0 if c == 0 else 0.8 for c in kind], top_k=[50 if c == 1 else 0 for c in kind],
               top_p=[0.9 if c == 2 else 1.0 for c in kind], min_p=[0.05 if c == 3 else 0.0 for c in kind])
    t.draw_noise(g)
    graph = t.capture()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    text, ms = [], 0.0
    for _ in range(a.steps):
        start.record()  # the noise of a step's draws is part of the step
        t.draw_noise(g)
        graph.replay()
        end.record()
        text.append(t.tokens.tolist())
        ms += start.elapsed_time(end)
    if bd.bd_get_device_status() != bd.BD_OK:
        raise RuntimeError(bd.bd_status_string(bd.bd_get_device_status()))
    for i in range(min(4, a.sequences)):
        print(f"sequence {i}, variant {ids[i]}: {[row[i] for row in text[:8]]} ...")
    print(f"{a.sequences} sequences, {a.layers} layers: {ms / a.steps:.3f} ms per step, "
          f"{a.sequences * a.steps / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
