"""Plain 64-bit forms of the decode-step operators, on the CPU, for the tests.

Written from the definitions in include/bitdelta.h; nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch


def randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float32) * std


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def rotated(x: np.ndarray, rope: np.ndarray) -> np.ndarray:
    """x [t, heads, dim], rope [t, dim] (cosines, sines)."""
    d = x.shape[-1] // 2
    c, s = rope[:, None, :d], rope[:, None, d:]
    a, b = x[..., :d], x[..., d:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def rotated_f32(x: torch.Tensor, rope: torch.Tensor) -> torch.Tensor:
    """The same with each product and sum rounded to fp32, as the cache write defines it."""
    d = x.shape[-1] // 2
    c, s = rope[:, None, :d], rope[:, None, d:]
    a, b = x.float()[..., :d], x.float()[..., d:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def quantised(x: torch.Tensor):
    """(e4m3 values, exponent bytes) of fp32 rows, by the definition of the 8-bit cache."""
    finite = torch.where(torch.isfinite(x), x, 0.0).double().abs().amax(-1).numpy()
    e = np.full(finite.shape, -60)
    on = finite > 0
    e[on] = np.clip(np.ceil(np.log2(finite[on] / 448)), -60, 120)
    # ceil(log2) is exact here: a bf16-derived maximum over 448 is a power of two only where log2 returns a whole number
    s = torch.from_numpy(2.0 ** e)[..., None]
    y = (x.double() / s).clamp(-448, 448).float()
    return y.to(torch.float8_e4m3fn), torch.from_numpy((e + 127).astype(np.uint8))


class Pool:
    """A paged cache built on the CPU: token values per sequence, pages in shuffled order."""

    def __init__(self, lengths, kv_heads, dim, page, kv, seed, spare=2, k_std=1.0, junk=None):
        rng = np.random.default_rng(seed)
        self.kv_heads, self.dim, self.page, self.kv, self.lengths = kv_heads, dim, page, kv, list(lengths)
        pages = [-(-n // page) for n in lengths]
        n_pages, width = sum(pages) + spare, max(1, max(pages, default=1))
        order, at = rng.permutation(n_pages), 0
        self.table = np.full((len(lengths), width), -1, np.int32)
        for i, p in enumerate(pages):
            self.table[i, :p] = order[at:at + p]
            at += p
        shape = (n_pages, kv_heads, page, dim)
        self.k, self.v = randn(shape, seed, k_std), randn(shape, seed + 1)
        if kv == "bf16":
            self.k, self.v = self.k.bfloat16(), self.v.bfloat16()
            self.k_scale = self.v_scale = None
        else:
            self.k, self.k_scale = quantised(self.k)
            self.v, self.v_scale = quantised(self.v)
        if junk is not None:  # every slot no token uses
            used = torch.zeros((n_pages, page), dtype=torch.bool)
            for i, n in enumerate(lengths):
                for t in range(n):
                    used[self.table[i, t // page], t % page] = True
            free = ~used[:, None, :].expand(-1, kv_heads, -1)
            for x in (self.k, self.v):
                raw = x.view(torch.uint8) if kv != "bf16" else x
                raw[free] = torch.tensor(junk, dtype=raw.dtype)
            if kv != "bf16":
                self.k_scale[free] = 255
                self.v_scale[free] = 255

    def device(self):
        return {n: (None if t is None else t.cuda()) for n, t in
                (("k", self.k), ("v", self.v), ("k_scale", self.k_scale), ("v_scale", self.v_scale))}

    def cache(self):
        from bit_delta_tenant_gb300 import bitdelta as bd
        return bd.KVCache(**self.device())

    def values(self, name, i, n=None):
        """Tokens of sequence i in 64 bits, [n, kv_heads, dim]."""
        n = self.lengths[i] if n is None else n
        t = np.arange(n)
        page, slot = self.table[i, t // self.page], t % self.page
        x = f64(getattr(self, name).float())[page, :, slot]
        if self.kv != "bf16":
            x = x * 2.0 ** (getattr(self, name + "_scale").numpy().astype(np.float64)[page, :, slot] - 127)[..., None]
        return x


def attention(q, k, v, scale):
    """q [heads, dim], k and v [n, kv_heads, dim] -> out, lse, and what the error bounds need:
    sum p |v| per output and the largest scale * sum |q k| per head."""
    heads, dim = q.shape
    n, kv_heads, _ = k.shape
    g = heads // kv_heads
    if n == 0:
        return np.zeros((heads, dim)), np.full(heads, -np.inf), np.zeros((heads, dim)), np.zeros(heads)
    qh = q.reshape(kv_heads, g, dim)
    s = np.einsum("hgd,nhd->hgn", qh, k) * scale
    big = (np.einsum("hgd,nhd->hgn", np.abs(qh), np.abs(k)) * abs(scale)).max(-1).reshape(heads)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(-1, keepdims=True)
    lse = (top + np.log(total)).reshape(heads)
    p = p / total
    out = np.einsum("hgn,nhd->hgd", p, v).reshape(heads, dim)
    mag = np.einsum("hgn,nhd->hgd", p, np.abs(v)).reshape(heads, dim)
    return out, lse, mag, big


def sample(x, noise, t, k, p, low):
    """(id, logprob) of one row; x and noise fp32.  z and z + noise are rounded as defined, weights are 64-bit."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float32)
    noise = np.where(np.isnan(noise), -np.inf, noise).astype(np.float32)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf
    greedy = not t > 0
    with np.errstate(all="ignore"):
        inv = np.float32(1) if greedy else np.float32(1) / np.float32(t)
        z = ((x - top).astype(np.float32) * inv).astype(np.float32)
        z = np.where(np.isnan(z), -np.inf, z)
        z[x == top] = 0
        w = np.exp(z.astype(np.float64))
        order = np.argsort(-x.astype(np.float64), kind="stable")
        order = order[x[order] > -np.inf]
        if greedy:
            order = order[:1]
        if k > 0:
            order = order[:k]
        if p <= 0:
            order = order[:1]
        elif p < 1:
            mass = np.cumsum(w[order])
            order = order[np.concatenate([[True], mass[:-1] < p * mass[-1]])]
        if low > 0:
            order = order[w[order] >= min(low, 1.0)]
        order = np.sort(order)
        score = (z + noise).astype(np.float32)
        score = np.where(np.isnan(score), -np.inf, score)
        i = int(order[0] if greedy else order[np.argmax(score[order])])
        return i, float(z[i]) - float(np.log(w[x > -np.inf].sum()))
