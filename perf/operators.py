"""Workloads of the decode-step operators around the fused linears.

Five operators of a multi-tenant decode step: the residual norm in front of a
linear, the rotary/quantising write into a paged key-value cache, reading that
cache back, the attention of one new token over it, and the draw of the next
token.  Each has a plain form in elementary torch operations (fp32, rounded
once at the end), the framework's call, and a definition in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

#: False: the plain forms; True: the framework's operators.
own = False

EPS = 1e-5
E4M3_MAX = 448.0
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the residual norm of one request's decode step: latency
        dict(name="norm: 1 x 4096", op="norm", m=1, n=4096, variants=1, residual=True, out="bf16"),
        # 64 tokens of 14 tenants, each with its own norm weights, handed on in 8 bits
        dict(name="norm: 64 x 8192, 14 variants, 8 bits", op="norm", m=64, n=8192, variants=14, residual=True, out="e4m3"),
        # a prefill batch
        dict(name="norm: 8192 x 8192", op="norm", m=8192, n=8192, variants=1, residual=True, out="bf16"),
        # one new token of each of 64 sequences
        dict(name="append: 64 tokens, 8 bits", op="append", seqs=64, new=1, past=1000, q_heads=32, kv_heads=8, dim=128,
             page=16, kv="e4m3"),
        # a chunk of prompts, 70B-shape heads
        dict(name="append: prompts up to 4096", op="append", seqs=8, new=4096, past=1, q_heads=64, kv_heads=8, dim=128,
             page=64, kv="e4m3"),
        # one prompt's cache read back
        dict(name="read: 1000 tokens", op="read", seqs=1, longest=1000, kv_heads=8, dim=128, page=16, kv="bf16"),
        # many sequences' caches moved out
        dict(name="read: 64 sequences, 8 bits", op="read", seqs=64, longest=8191, kv_heads=8, dim=128, page=32, kv="e4m3"),
        # one request's decode step over a short context: latency
        dict(name="attention: 1 x 777", op="attention", seqs=1, longest=777, q_heads=32, kv_heads=8, dim=128, page=16,
             kv="bf16", window=0),
        # a full decode batch of ragged lengths, one slot empty
        dict(name="attention: 64 ragged, 8 bits", op="attention", seqs=64, longest=8191, q_heads=32, kv_heads=8, dim=128,
             page=32, kv="e4m3", window=0),
        # one long document, 70B-shape heads
        dict(name="attention: 1 x 130001", op="attention", seqs=1, longest=130001, q_heads=64, kv_heads=8, dim=128, page=64,
             kv="bf16", window=0),
        # the next token of one request
        dict(name="sample: 1 row", op="sample", m=1, vocab=128256, logits="bf16", filters="k+p"),
        # the next token of a batch, each row with its own settings
        dict(name="sample: 256 rows, mixed", op="sample", m=256, vocab=128256, logits="f32", filters="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "read", "attention", "sample"])
    kv, page, dim = rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    q_heads, kv_heads = rng.choice([(32, 8), (32, 32), (64, 8), (8, 1), (12, 4), (16, 16), (48, 4)])
    if op == "norm":
        n = 8 * _log(rng, 64, 1792)
        out = rng.choice(["bf16", "e4m3"])
        n = -(-n // 128) * 128 if out == "e4m3" else n
        return dict(op=op, m=_log(rng, 1, max(1, min(16384, (8192 * 8192) // n))), n=n, variants=rng.choice([1, 3, 14]),
                    residual=rng.random() < 0.8, out=out)
    if op == "append":
        seqs, new = _log(rng, 1, 256), rng.choice([1, 1, _log(rng, 2, 4096)])
        while seqs * new * (q_heads + 2 * kv_heads) * dim > 8000 * 80 * 128:
            seqs, new = max(1, seqs // 2), max(1, new // 2)
        return dict(op=op, seqs=seqs, new=new, past=_log(rng, 1, 1000), q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page,
                    kv=kv)
    if op == "sample":
        return dict(op=op, m=_log(rng, 1, 256), vocab=_log(rng, 1000, 128256), logits=rng.choice(["bf16", "f32"]),
                    filters=rng.choice(["none", "k", "p", "k+p", "min-p", "greedy", "mixed"]))
    seqs, longest = _log(rng, 1, 256), _log(rng, 1, 130000)
    while seqs * longest * kv_heads * dim > (130000 if op == "attention" else 65000) * 8 * 128:  # a read moves twice as much
        seqs, longest = max(1, seqs // 2), max(1, longest * 2 // 3)
    c = dict(op=op, seqs=seqs, longest=longest, kv_heads=kv_heads, dim=dim, page=page, kv=kv)
    if op == "attention":
        c.update(q_heads=q_heads, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    return c


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, even in their logarithm; hi is one of them."""
    return [hi if i == n - 1 else int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _lengths(c):
    """The sequences' lengths; a batch of 8 and more has an empty slot."""
    v = _spread(c["seqs"], 1, c["longest"])
    return [0] + v[1:] if len(v) >= 8 else v


def work(c):
    if c["op"] == "norm":
        e = c["m"] * c["n"]
        by = 2 * e + (4 * e if c["residual"] else 0) + 2 * min(c["m"], c["variants"]) * c["n"]
        by += 2 * e if c["out"] == "bf16" else e + 4 * (e // 128)
        return {"bytes": by, "flops": 6 * e}
    size = lambda c: c["dim"] * (2 if c["kv"] == "bf16" else 1) + (0 if c["kv"] == "bf16" else 1)  # noqa: E731
    if c["op"] == "append":
        t = sum(_spread(c["seqs"], 1, c["new"]))
        row = 2 * c["dim"]
        return {"bytes": t * (2 * c["q_heads"] * row + 2 * c["kv_heads"] * (row + size(c)) + 4 * c["dim"] + 8),
                "flops": t * 6 * (c["q_heads"] + c["kv_heads"]) * c["dim"]}
    if c["op"] == "read":
        t = sum(_lengths(c))
        return {"bytes": 2 * t * c["kv_heads"] * (size(c) + 2 * c["dim"]), "flops": 2 * t * c["kv_heads"] * c["dim"]}
    if c["op"] == "attention":
        t = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
        return {"bytes": 2 * t * c["kv_heads"] * size(c) + 4 * c["seqs"] * c["q_heads"] * c["dim"],
                "flops": 4 * t * c["q_heads"] * c["dim"]}
    free = {"none": c["m"], "mixed": -(-c["m"] // 6)}.get(c["filters"], 0)  # rows that need all of their noise
    return {"bytes": c["m"] * c["vocab"] * (2 if c["logits"] == "bf16" else 4) + 4 * free * c["vocab"],
            "flops": 4 * c["m"] * c["vocab"]}


# ---------------------------------------------------------------- inputs

def _randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _scales(x):
    """Exponent byte (bias 127) of the smallest power of two s >= 2^-60 with max|x| / s <= 448, over the last axis."""
    m, e = torch.frexp(x.abs().amax(-1))
    return torch.where(m > 0, e - torch.where(m <= 0.875, 9, 8), -60).clamp(-60, 120) + 127


def _power(byte):
    return torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.to(torch.int32) - 127)


def _e4m3(x):
    """(values in e4m3, exponent bytes of their scales) of rows x."""
    b = _scales(x)
    return (x / _power(b)[..., None]).to(torch.float8_e4m3fn), b.to(torch.uint8)


def _cache(c, lens, g, rng):
    """A pool of pages whose order is shuffled, and each sequence's table of them."""
    pages = [-(-n // c["page"]) for n in lens]
    total, width = max(1, sum(pages)) + 3, max(1, max(pages))
    order, at = rng.permutation(total), 0
    table = np.full((len(lens), width), -1, np.int32)
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p]
        at += p
    shape = (total, c["kv_heads"], c["page"], c["dim"])
    s = {"table": torch.from_numpy(table).to(DEV), "k_scale": None, "v_scale": None}
    # a few channels of K are several times larger than the rest
    gain = torch.ones(c["dim"], device=DEV)
    gain[3::29] = 4.0
    for name, mul in (("k", gain), ("v", 0.5)):
        x = _randn(shape, g).mul_(mul)
        if c["kv"] == "bf16":
            s[name] = x.to(torch.bfloat16)
        else:
            s[name], s[name + "_scale"] = _e4m3(x)
    return s


def _rope(n, dim):
    """cos | sin of position p and pair i, fp32 [n, dim]."""
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(dim // 2) / (dim // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    ints = lambda v: torch.from_numpy(np.asarray(v, np.int32)).to(DEV)  # noqa: E731
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if c["op"] == "norm":
        m, n = c["m"], c["n"]
        s = {"x": _randn((m, n), g).to(torch.bfloat16), "weight": _randn((c["variants"], n), g, 0.1).add_(1).to(torch.bfloat16),
             "ids": ints(rng.randint(0, c["variants"], m)) if c["variants"] > 1 else None, "residual": None, "residual_out": None}
        if c["residual"]:
            s["residual"] = _randn((m, n), g, 3.0).to(torch.bfloat16)
            s["residual_out"] = torch.empty((m, n), **bf16)
        s["y"] = torch.empty((m, n), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float8_e4m3fn, device=DEV)
        s["y_scale"] = None if c["out"] == "bf16" else torch.empty((m, n // 128), dtype=torch.float32, device=DEV)
    elif c["op"] == "append":
        new, past = _spread(c["seqs"], 1, c["new"]), _spread(c["seqs"], 1, c["past"])
        rng.shuffle(new), rng.shuffle(past)
        s = _cache(c, [a + b for a, b in zip(new, past)], g, rng)
        t = sum(new)
        s["seq_ids"] = ints(np.repeat(np.arange(c["seqs"]), new))
        s["positions"] = ints(np.concatenate([np.arange(b, b + a) for a, b in zip(new, past)]))
        s["rope"] = _rope(c["new"] + c["past"] + 1, c["dim"])
        s["q_out"] = torch.empty((t, c["q_heads"], c["dim"]), **bf16)
        for name, heads in (("q", c["q_heads"]), ("new_k", c["kv_heads"]), ("new_v", c["kv_heads"])):
            s[name] = _randn((t, heads, c["dim"]), g).to(torch.bfloat16)
    elif c["op"] == "read":
        lens = _lengths(c)
        rng.shuffle(lens)
        s = _cache(c, lens, g, rng)
        s["offsets"] = ints(np.concatenate([[0], np.cumsum(lens)]))
        s["k_out"], s["v_out"] = (torch.empty((sum(lens), c["kv_heads"], c["dim"]), **bf16) for _ in "kv")
    elif c["op"] == "attention":
        lens = _lengths(c)
        rng.shuffle(lens)
        s = _cache(c, lens, g, rng)
        s["lengths"] = ints(lens)
        s["q"] = _randn((c["seqs"], c["q_heads"], c["dim"]), g, 1.5).to(torch.bfloat16)
        s["out"] = torch.empty((c["seqs"], c["q_heads"], c["dim"]), **bf16)
        s["lse"] = torch.empty((c["seqs"], c["q_heads"]), dtype=torch.float32, device=DEV)
    else:
        m, v = c["m"], c["vocab"]
        # logits fall off with the logarithm of their rank, as a language model's do
        rank = torch.rand((m, v), generator=g, device=DEV).mul_(v - 1).add_(1)
        x = rank.log_().mul_(-1.3).add_(_randn((m, v), g, 0.7)).add_(9.0)
        s = {"logits": x.to(torch.bfloat16) if c["logits"] == "bf16" else x}
        u = torch.rand((m, v), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
        s["noise"] = u.log_().neg_().log_().neg_()
        f = {"none": [0], "k": [1], "p": [2], "k+p": [3], "min-p": [4], "greedy": [5], "mixed": [0, 1, 2, 3, 4, 5]}[c["filters"]]
        f = np.array([f[i % len(f)] for i in range(m)])
        r = rng.rand(m).astype(np.float32)
        s["temperature"] = torch.from_numpy(np.where(f == 5, 0, 0.6 + 0.8 * r).astype(np.float32)).to(DEV)
        s["top_k"] = ints(np.where((f == 1) | (f == 3), rng.randint(20, 200, m), 0))
        s["top_p"] = torch.from_numpy(np.where((f == 2) | (f == 3), 0.8 + 0.15 * r, 1).astype(np.float32)).to(DEV)
        s["min_p"] = torch.from_numpy(np.where(f == 4, 0.02 + 0.1 * r, 0).astype(np.float32)).to(DEV)
        s["ids"] = torch.empty((m,), dtype=torch.int32, device=DEV)
        s["logprob"] = torch.empty((m,), dtype=torch.float32, device=DEV)
    s["case"] = c
    return s


# ---------------------------------------------------------------- plain forms

def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    w = s["weight"].float()
    w = w[s["ids"].long()] if s["ids"] is not None else w[0]
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w
    out = {} if s["residual"] is None else {"residual": h.to(torch.bfloat16)}
    if s["y_scale"] is None:
        return {"y": y.to(torch.bfloat16), **out}
    b = y.view(y.shape[0], -1, 128)
    top = b.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    return {"y": (b * (1 / scale)[..., None]).to(torch.float8_e4m3fn).view_as(y), "scale": scale, **out}


def _plain_append(s):
    cos, sin = s["rope"][s["positions"].long()][:, None].chunk(2, -1)

    def rotated(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    page = s["k"].shape[2]
    at = s["positions"].long()
    pages = s["table"][s["seq_ids"].long(), at // page].long()
    for name, x in (("k", rotated(s["new_k"])), ("v", s["new_v"].float())):
        if s["k_scale"] is None:
            s[name][pages, :, at % page] = x.to(torch.bfloat16)
        else:
            x, b = _e4m3(x)
            s[name].view(torch.uint8)[pages, :, at % page] = x.view(torch.uint8)
            s[name + "_scale"][pages, :, at % page] = b
    return _appended(s, rotated(s["q"]).to(torch.bfloat16))


def _appended(s, q):
    out = {"q": q, "k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:  # the bytes are powers of two: the type says so
        out.update(k_scale=s["k_scale"].view(torch.float8_e8m0fnu), v_scale=s["v_scale"].view(torch.float8_e8m0fnu))
    return out


def _rows(s, name, index):
    """Rows of the pool as fp32, the index over (page, head, slot)."""
    if s["k_scale"] is None:
        return s[name][index].float()
    return s[name].view(torch.uint8)[index].view(torch.float8_e4m3fn).float() * _power(s[name + "_scale"][index])[..., None]


def _plain_read(s):
    total, page = s["k_out"].shape[0], s["k"].shape[2]
    t = torch.arange(total, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"], t, right=True) - 1
    at = (t - s["offsets"][seq]).long()
    index = (s["table"][seq, at // page].long(), slice(None), at % page)
    return {"k": _rows(s, "k", index).to(torch.bfloat16), "v": _rows(s, "v", index).to(torch.bfloat16)}


def _plain_attention(s):
    n, heads, dim = s["q"].shape
    _, kv_heads, page, _ = s["k"].shape
    at = torch.arange(s["table"].shape[1] * page, device=DEV)
    seen = at < s["lengths"][:, None]
    if s["case"]["window"]:
        seen &= at >= s["lengths"][:, None] - s["case"]["window"]
    index = (s["table"].clamp(min=0).long(),)
    k, v = (_rows(s, name, index).transpose(1, 2).reshape(n, kv_heads, -1, dim) for name in "kv")
    v = torch.where(seen[:, None, :, None], v, 0.0)
    x = s["q"].float().view(n, kv_heads, heads // kv_heads, dim) @ k.transpose(-1, -2) * (1 / math.sqrt(dim))
    x = torch.where(seen[:, None, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, p @ v / total, 0.0)
    return {"out": out.view(n, heads, dim).to(torch.bfloat16), "lse": (top + torch.log(total)).view(n, heads)}


def _plain_sample(s):
    x, at = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    t = s["temperature"][:, None]
    k, p = s["top_k"][:, None], s["top_p"][:, None]
    z = (x - x[:, :1]) * torch.where(t > 0, 1 / t, 1.0)
    w = torch.exp(z)
    rank = torch.arange(x.shape[1], device=DEV)
    keep = (rank < torch.where(k > 0, k, x.shape[1])) & ((t > 0) | (rank == 0))
    kept = torch.where(keep, w, 0.0)
    keep &= (kept.cumsum(-1) - kept < p * kept.sum(-1, keepdim=True)) | (p >= 1)
    keep &= w >= s["min_p"][:, None]
    score = torch.where(keep, z + s["noise"].gather(1, at), -torch.inf)
    ids = torch.empty_like(score).scatter_(1, at, score).argmax(-1)
    zid = torch.empty_like(z).scatter_(1, at, z).gather(1, ids[:, None])[:, 0]
    return {"ids": ids.to(torch.int32), "logprob": zid - torch.log(w.sum(-1))}


# ---------------------------------------------------------------- one pass

def _own(s):
    from bit_delta_tenant_gb300 import bitdelta as bd

    op = s["case"]["op"]
    if op == "norm":
        bd.bd_rmsnorm(s["x"], s["weight"], EPS, s["y"], residual=s["residual"], residual_out=s["residual_out"],
                      y_scale=s["y_scale"], weight_ids=s["ids"])
        out = {"y": s["y"]}
        if s["residual"] is not None:
            out["residual"] = s["residual_out"]
        if s["y_scale"] is not None:
            out["scale"] = s["y_scale"]
        return out
    if op == "sample":
        bd.bd_sample(s["logits"], s["noise"], s["ids"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], logprob=s["logprob"])
        return {"ids": s["ids"], "logprob": s["logprob"]}
    cache = s.get("cache")
    if cache is None:  # a program keeps the cache's handle
        cache = s["cache"] = bd.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op == "append":
        bd.bd_kv_append(cache, s["q"], s["new_k"], s["new_v"], s["positions"], s["table"], s["rope"], s["q_out"],
                        seq_ids=s["seq_ids"])
        return _appended(s, s["q_out"])
    if op == "read":
        bd.bd_kv_read(cache, s["table"], s["offsets"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if "workspace" not in s:  # and one zero-filled workspace
        need = bd.bd_attention_workspace_size(cache, s["q"].shape[0], s["q"].shape[1])
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    bd.bd_attention_decode(cache, s["q"], s["table"], s["lengths"], s["out"], s["workspace"],
                           scale=1 / math.sqrt(s["case"]["dim"]), window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


_PLAIN = {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "attention": _plain_attention, "sample": _plain_sample}


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


# ---------------------------------------------------------------- the definitions in 64 bits

def _host(t):
    return t.double().cpu().numpy()


def _round_e4m3(x):
    """Nearest e4m3 number (ties to even) of each |x| <= 464, in 64 bits."""
    step = 2.0 ** (np.clip(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))), -6, 8) - 3)
    return np.clip(np.round(x / step) * step, -448, 448)


def _stored(s, name):
    """The pool's values in 64 bits, [page, head, slot, dim] on the device."""
    x = s[name].double()
    return x if s["k_scale"] is None else x * torch.exp2(s[name + "_scale"].double() - 127)[..., None]


def _exact_norm(s):
    h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    w = s["weight"].double()
    w = w[0] if s["ids"] is None else w.index_select(0, s["ids"])
    y = w * (h / (h.pow(2).sum(1) / h.shape[1] + EPS).sqrt()[:, None])
    out = {} if s["residual"] is None else {"residual": h}
    if s["y_scale"] is None:
        return {"y": y, **out}
    y = y.cpu().numpy().reshape(h.shape[0], -1, 128)
    scale = np.abs(y).max(2) / 448
    return {"y": _round_e4m3(y / scale[:, :, None]).reshape(h.shape), "scale": scale, **{k: v.cpu().numpy() for k, v in out.items()}}


def _exact_append(s):
    pos, seq, table = (s[k].cpu().numpy().astype(np.int64) for k in ("positions", "seq_ids", "table"))
    d = s["q"].shape[2] // 2
    angle = _host(s["rope"])[pos]
    turn = (angle[:, :d] + 1j * angle[:, d:])[:, None]

    def rotated(x):
        x = _host(x)
        z = (x[:, :, :d] + 1j * x[:, :, d:]) * turn
        return np.concatenate([z.real, z.imag], 2)

    page = s["k"].shape[2]
    where = (table[seq, pos // page], slice(None), pos % page)
    out = {"q": rotated(s["q"])}
    for name, x in (("k", rotated(s["new_k"])), ("v", _host(s["new_v"]))):
        pool = s[name].float().cpu().numpy()
        if s["k_scale"] is None:
            pool[where] = x
        else:
            low = np.ceil(np.log2(np.maximum(np.abs(x).max(2), 1e-300) / 448)).clip(-60, 120)
            pool[where] = _round_e4m3(x / 2.0 ** low[:, :, None])
            scale = 2.0 ** (s[name + "_scale"].cpu().numpy().astype(np.float64) - 127)
            scale[where] = 2.0 ** low
            out[name + "_scale"] = scale
        out[name] = pool
    return out


def _tokens(s, i, n):
    """(page, slot) of the first n tokens of sequence i."""
    t = torch.arange(n, device=DEV)
    page = s["k"].shape[2]
    return s["table"][i].long().index_select(0, t.div(page, rounding_mode="floor")), t.remainder(page)


def _exact_read(s):
    ends = s["offsets"].tolist()
    out = {}
    for name in "kv":
        x = _stored(s, name)
        out[name] = torch.cat([x[p, :, t] for p, t in (_tokens(s, i, b - a) for i, (a, b) in enumerate(zip(ends, ends[1:])))])
    return out


def _exact_attention(s):
    n, heads, dim = s["q"].shape
    kv_heads, window = s["k"].shape[1], s["case"]["window"]
    out, lse = torch.zeros((n, heads, dim), dtype=torch.float64, device=DEV), torch.full((n, heads), -torch.inf, dtype=torch.float64, device=DEV)
    ks, vs = _stored(s, "k"), _stored(s, "v")
    for i, length in enumerate(s["lengths"].tolist()):
        if not length:
            continue
        p, t = _tokens(s, i, length)
        if window:
            p, t = p[-window:], t[-window:]
        q = s["q"][i].double().view(kv_heads, -1, dim)
        x = torch.einsum("hgd,thd->hgt", q, ks[p, :, t]) / math.sqrt(dim)
        lse[i] = torch.logsumexp(x, -1).view(-1)
        out[i] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), vs[p, :, t]).reshape(heads, dim)
    return {"out": out, "lse": lse}


def _exact_sample(s):
    logits, noise = _host(s["logits"]), _host(s["noise"])
    ids, logprob = [], []
    for x, g, t, k, p, low in zip(logits, noise, *(s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p"))):
        z = (x - x.max()) / (t if t > 0 else 1)
        w = np.exp(z)
        order = np.argsort(-x, kind="stable")
        if t <= 0:
            order = order[:1]
        elif k > 0:
            order = order[:k]
        if p < 1:
            mass = np.cumsum(w[order])
            order = order[: 1 + int(np.searchsorted(mass[:-1], p * mass[-1]))]
        order = np.sort(order[w[order] >= low])
        ids.append(order[np.argmax(z[order] + g[order])])
        logprob.append(z[ids[-1]] - np.log(w.sum()))
    return {"ids": np.array(ids, np.int32), "logprob": np.array(logprob)}


def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "append": _exact_append, "read": _exact_read, "attention": _exact_attention, "sample": _exact_sample}[c["op"]](s)
