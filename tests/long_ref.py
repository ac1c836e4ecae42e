"""Plain 64-bit forms of the long-context operators, on the CPU, for the tests.

Written from the definitions in include/bitdelta.h; nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

from step_ref import f64, quantised, randn

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LEVELS = np.array([m * 2.0 ** -17 for m in range(8)] + [2.0 ** (b // 8 - 15) * (1 + b % 8 / 8) for b in range(8, 248)])


def nearest(x, table):
    """Index of the entry of an ascending table nearest to each x >= 0, ties to even indices, beyond the last to it."""
    i = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo, hi = x - table[i - 1], table[i] - x
    return np.where((lo < hi) | ((lo == hi) & ((i - 1) % 2 == 0)), i - 1, i)


def four_bits(x: torch.Tensor):
    """(bytes of two 4-bit codes, scale bytes) of fp32 rows, by the definition of the 4-bit cache."""
    g = x.numpy().astype(np.float64).reshape(*x.shape[:-1], -1, 16)
    top = np.where(np.isfinite(g), np.abs(g), 0).max(-1)
    b = nearest((top.astype(np.float32) / np.float32(6)).astype(np.float64), LEVELS)
    s = LEVELS[b][..., None]
    with np.errstate(all="ignore"):
        y = np.abs((g.astype(np.float32) / s.astype(np.float32)).astype(np.float64))
    code = nearest(np.minimum(np.where((s > 0) & ~np.isnan(y), y, 0), 6), CODES) + 8 * np.signbit(g)
    code = code.reshape(x.shape).astype(np.uint8)
    b = np.where(np.isnan(g).any(-1), 255, b).astype(np.uint8)
    return torch.from_numpy(code[..., 0::2] | code[..., 1::2] << 4), torch.from_numpy(b)


def four_values(raw: np.ndarray, scale: np.ndarray) -> np.ndarray:
    code = np.stack([raw & 15, raw >> 4], -1).reshape(*raw.shape[:-1], 2 * raw.shape[-1])
    x = CODES[code & 7] * np.where(code & 8, -1.0, 1.0)
    level = np.concatenate([LEVELS, [np.inf], np.full(7, np.nan)])
    with np.errstate(all="ignore"):
        return x * np.repeat(level[scale], 16, -1)


class Pool:
    """A paged cache built on the CPU: bf16, e4m3 or e2m1, pages in shuffled order, `junk` in the slots no token uses."""

    def __init__(self, lengths, kv_heads, dim, page, kv, seed, spare=2, k_std=1.0, junk=False):
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
        self.set("k", randn(shape, seed, k_std)), self.set("v", randn(shape, seed + 1))
        if junk:
            used = torch.zeros((n_pages, page), dtype=torch.bool)
            for i, n in enumerate(lengths):
                t = np.arange(n)
                used[self.table[i, t // page], t % page] = True
            self.spoil(~used[:, None, :].expand(-1, kv_heads, -1))

    def set(self, name, x):
        scale = None
        if self.kv == "bf16":
            x = x.bfloat16()
        elif self.kv == "e4m3":
            x, scale = quantised(x)
        else:
            x, scale = four_bits(x)
        setattr(self, name, x), setattr(self, name + "_scale", scale)

    def spoil(self, where):
        """NaN in K and V of the slots [n_pages, kv_heads, page]."""
        for name in "kv":
            if self.kv == "bf16":
                getattr(self, name)[where] = float("nan")
            else:
                getattr(self, name).view(torch.uint8)[where] = 0x7F
                getattr(self, name + "_scale")[where] = 255

    def spoil_tokens(self, i, tokens):
        where = torch.zeros((self.k.shape[0], self.page), dtype=torch.bool)
        t = np.asarray(tokens)
        where[self.table[i, t // self.page], t % self.page] = True
        self.spoil(where[:, None, :].expand(-1, self.kv_heads, -1))

    def cache(self):
        from bit_delta_tenant_gb300 import bitdelta as bd
        return bd.KVCache(*(None if t is None else t.cuda() for t in (self.k, self.v, self.k_scale, self.v_scale)))

    def values(self, name, i, n=None):
        """Tokens of sequence i in 64 bits, [n, kv_heads, dim]."""
        n = self.lengths[i] if n is None else n
        t = np.arange(n)
        at = (self.table[i, t // self.page], slice(None), t % self.page)
        if self.kv == "e2m1":
            return four_values(getattr(self, name).numpy()[at], getattr(self, name + "_scale").numpy()[at])
        x = f64(getattr(self, name).float())[at]
        if self.kv == "e4m3":
            with np.errstate(all="ignore"):
                x = x * 2.0 ** (getattr(self, name + "_scale").numpy().astype(np.float64)[at] - 127)[..., None]
        return x


def attention(q, k, v, p, scale, window=0, cap=0.0, slopes=None, first=0, prefix=0):
    """One query q [heads, dim] at position p over k and v [n, kv_heads, dim]: out, lse, and what error bounds need: the sum
    of p |v| per output, and the largest |score| before and after the rule per head."""
    heads, dim = q.shape
    n, kv_heads, _ = k.shape
    j = np.arange(n)
    seen = ((j <= p) | (j < prefix)) & (j >= first)
    if window:
        seen &= j > p - window
    if p < 0 or not seen.any():
        return np.zeros((heads, dim)), np.full(heads, -np.inf), np.zeros((heads, dim)), np.zeros(heads)
    k, v, j = k[seen], v[seen], j[seen]
    qh = q.reshape(kv_heads, heads // kv_heads, dim)
    s = np.einsum("hgd,nhd->hgn", qh, k) * scale
    big = (np.einsum("hgd,nhd->hgn", np.abs(qh), np.abs(k)) * abs(scale)).max(-1).reshape(heads)
    if cap:
        s = cap * np.tanh(s / cap)
    if slopes is not None:
        far = slopes.reshape(kv_heads, -1, 1) * np.abs(p - j)
        s = s - far
        big = big + np.abs(far).max(-1).reshape(heads)
    top = s.max(-1, keepdims=True)
    w = np.exp(s - top)
    total = w.sum(-1, keepdims=True)
    w = w / total
    out = np.einsum("hgn,nhd->hgd", w, v).reshape(heads, dim)
    mag = np.einsum("hgn,nhd->hgd", w, np.abs(v)).reshape(heads, dim)
    return out, (top + np.log(total)).reshape(heads), mag, big
