"""Workloads of the operators for long contexts beside the fused linears.

The attention of whole prompts over a paged key-value cache, and of single new
tokens, with scores that are capped or biased by distance and with window,
document and prefix masks; a cache held in 4 bits (rotated and quantised as it
is written, read back, attended to); and the table of rotary positions, scaled
for contexts longer than a model was trained on.  Each has a plain form in
elementary torch operations (fp32, rounded once at the end), the framework's
call, and a definition in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

#: False: the plain forms; True: the framework's operators.
own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    heads = dict(q_heads=32, kv_heads=8, dim=128)
    plain = dict(window=0, cap=0.0, slopes=False, docs=0, prefix=False)
    return [
        # the positions of a short context, no scaling
        dict(name="table: 4096 x 64", op="table", positions=4096, dim=64, factor=1.0, original=0, amplitude=1.0),
        # a context 16 times as long as the one trained on
        dict(name="table: 131072 x 128, scaled", op="table", positions=131072, dim=128, factor=16.0, original=8192, amplitude=1.28),
        # one new token of each of 64 sequences, half of each head rotated, and their last tokens read back
        dict(name="store: 64 tokens", op="store", seqs=64, new=1, past=40, page=16, rotated=64, interleaved=True, **heads),
        # a chunk of prompts, 70B-shape heads, written and read back
        dict(name="store: prompts up to 4096", op="store", seqs=8, new=4096, past=1, page=64, rotated=128, interleaved=False,
             q_heads=64, kv_heads=8, dim=128),
        # one request's decode step over a short context, capped scores: latency
        dict(name="token: 1 x 777, capped", op="token", seqs=1, longest=777, page=16, kv="bf16", **heads, **{**plain, "cap": 50.0}),
        # a full decode batch of ragged lengths, 4 bits, scores biased by distance
        dict(name="token: 64 ragged, 4 bits", op="token", seqs=64, longest=8191, page=32, kv="e2m1", **heads,
             **{**plain, "slopes": True}),
        # one long document in 4 bits, 70B-shape heads
        dict(name="token: 1 x 130001, 4 bits", op="token", seqs=1, longest=130001, page=64, kv="e2m1", q_heads=64, kv_heads=8,
             dim=128, **plain),
        # a short prompt: latency
        dict(name="prompt: 1 x 333", op="prompt", seqs=1, new=333, past=0, page=16, kv="bf16", **heads, **plain),
        # a long prompt
        dict(name="prompt: 1 x 8192", op="prompt", seqs=1, new=8192, past=0, page=64, kv="bf16", **heads, **plain),
        # ragged chunks of several requests over what is cached in 8 bits, capped, a prefix that sees itself whole
        dict(name="prompt: 9 ragged, 8 bits", op="prompt", seqs=9, new=1500, past=1000, page=32, kv="e4m3", **heads,
             **{**plain, "cap": 30.0, "prefix": True}),
        # a few tokens more of a long document in 4 bits
        dict(name="prompt: 48 over 65000, 4 bits", op="prompt", seqs=1, new=48, past=65000, page=64, kv="e2m1", q_heads=64,
             kv_heads=8, dim=128, **plain),
        # documents packed into long sequences, small heads, scores biased by distance, a window
        dict(name="prompt: packed documents", op="prompt", seqs=2, new=6000, past=0, page=64, kv="bf16", q_heads=12, kv_heads=4,
             dim=64, **{**plain, "slopes": True, "docs": 11, "window": 1024}),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["table", "store", "token", "prompt", "prompt"])
    if op == "table":
        scaled = rng.random() < 0.7
        return dict(op=op, positions=_log(rng, 1, 131072), dim=rng.choice([16, 32, 64, 96, 128]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]) if scaled else 1.0,
                    original=rng.choice([0, 2048, 8192]) if scaled else 0, amplitude=rng.choice([1.0, 1.1, 1.4]))
    page, dim = rng.choice([16, 32, 48, 64, 128]), rng.choice([64, 128, 128])
    q_heads, kv_heads = rng.choice([(32, 8), (32, 32), (64, 8), (8, 1), (12, 4), (16, 16), (48, 4)])
    heads = dict(q_heads=q_heads, kv_heads=kv_heads, dim=dim)
    if op == "store":
        seqs, new = _log(rng, 1, 256), rng.choice([1, 1, _log(rng, 2, 4096)])
        past = _log(rng, 1, 1000)
        while seqs * (new + past) * (q_heads + 2 * kv_heads) * dim > 8000 * 80 * 128:
            seqs, new, past = max(1, seqs // 2), max(1, new * 2 // 3), max(1, past * 2 // 3)
        return dict(op=op, seqs=seqs, new=new, past=past, page=page, rotated=rng.choice([dim, dim, dim // 2, dim // 4]),
                    interleaved=rng.random() < 0.5, **heads)
    shape = dict(window=rng.choice([0, 0, _log(rng, 1, 4096)]), cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.4,
                 docs=0, prefix=False)
    kv = rng.choice(["bf16", "e4m3", "e2m1"])
    if op == "token":
        if kv != "e2m1" and not shape["slopes"]:
            shape["cap"] = 30.0
        seqs, longest = _log(rng, 1, 256), _log(rng, 1, 130000)
        while seqs * longest * kv_heads * dim > 130000 * 8 * 128:
            seqs, longest = max(1, seqs // 2), max(1, longest * 2 // 3)
        return dict(op=op, seqs=seqs, longest=longest, page=page, kv=kv, **heads, **shape)
    seqs, new, past = _log(rng, 1, 24), _log(rng, 1, 8000), rng.choice([0, 0, _log(rng, 1, 60000)])
    while seqs * new * (new + past) * q_heads > 8192 * 8192 * 16:
        seqs, new, past = max(1, seqs // 2), max(1, new * 2 // 3), past * 2 // 3
    shape["docs"], shape["prefix"] = rng.choice([0, 0, min(new, _log(rng, 2, 40))]), rng.random() < 0.3
    return dict(op=op, seqs=seqs, new=new, past=past, page=page, kv=kv, **heads, **shape)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, even in their logarithm; hi is one of them."""
    return [hi if i == n - 1 else int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _ragged(n, hi):
    """n lengths up to hi; a batch of 8 and more has an empty slot."""
    v = _spread(n, 1, hi) if hi else [0] * n
    return [0] + v[1:] if n >= 8 else v


def _prompts(c):
    """Of each sequence: new tokens, all tokens, the prefix's length; of each new token: the first position it sees."""
    rng = np.random.RandomState(7)
    new, past = _ragged(c["seqs"], c["new"]), _ragged(c["seqs"], c["past"])
    rng.shuffle(past)
    prefix, first = [], []
    for n, p in zip(new, past):
        prefix.append(int(rng.randint(0, n + p + 1)) // 2 if c["prefix"] else 0)
        if c["docs"]:
            at = np.arange(p, p + n)
            starts = np.sort(np.r_[0, rng.randint(0, max(1, n + p), c["docs"])])
            f = starts[np.searchsorted(starts, at, side="right") - 1]
            f[rng.rand(n) < 0.01] = 1 << 30  # a token between two documents sees nothing
            first.append(f)
    return new, [a + b for a, b in zip(new, past)], prefix, np.concatenate(first) if c["docs"] else None


def _sees(c):
    """Positions that the queries see, in all, and cached positions that some query sees."""
    if c["op"] == "token":
        t = sum(min(n, c["window"]) if c["window"] else n for n in _ragged(c["seqs"], c["longest"]))
        return t, t
    new, lens, prefix, first = _prompts(c)
    pairs = keys = at = 0
    for n, length, pre in zip(new, lens, prefix):
        p = np.arange(length - n, length)
        lo = np.maximum(0, p + 1 - c["window"]) if c["window"] else np.zeros_like(p)
        if first is not None:
            lo = np.maximum(lo, first[at:at + n])
        hi = np.maximum(p + 1, pre)
        pairs += int(np.maximum(0, hi - lo).sum())
        some = hi > lo
        keys += int(hi[some].max() - lo[some].min()) if some.any() else 0
        at += n
    return pairs, keys


def work(c):
    if c["op"] == "table":
        return {"bytes": 4 * c["positions"] * c["dim"], "flops": 20 * c["positions"] * c["dim"]}
    size = {"bf16": 2 * c["dim"], "e4m3": c["dim"] + 1, "e2m1": c["dim"] // 2 + c["dim"] // 16}[c.get("kv", "e2m1")]
    if c["op"] == "store":
        new, past = sum(_spread(c["seqs"], 1, c["new"])), sum(_spread(c["seqs"], 1, c["past"]))
        row = 2 * c["dim"]
        return {"bytes": new * (2 * c["q_heads"] * row + 2 * c["kv_heads"] * (row + size) + 4 * c["rotated"] + 8)
                + (new + past) * 2 * c["kv_heads"] * (size + row),
                "flops": new * 6 * (c["q_heads"] + c["kv_heads"]) * c["dim"] + 4 * (new + past) * c["kv_heads"] * c["dim"]}
    pairs, keys = _sees(c)
    rows = c["seqs"] if c["op"] == "token" else sum(_prompts(c)[0])
    return {"bytes": 2 * keys * c["kv_heads"] * size + 4 * rows * c["q_heads"] * c["dim"], "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------- the formats

def _randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _e4m3(x):
    """Rows x as e4m3 values and exponent bytes (bias 127): the smallest power of two s >= 2^-60 with max|x| / s <= 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    b = torch.where(m > 0, e - torch.where(m <= 0.875, 9, 8), -60).clamp(-60, 120)
    return torch.ldexp(x, -b[..., None]).to(torch.float8_e4m3fn), (b + 127).to(torch.uint8)


def _level(b):
    """Values of 4-bit scale bytes: 5 bits of exponent and 3 of mantissa, an fp16 number's bits 7 to 14."""
    return (b.to(torch.int16) << 7).view(torch.float16).float()


def _e2m1(x):
    """Rows x in 4 bits: bytes of two values each (the first in the low half) and a scale byte for each 16 values.

    The scale is the group's largest magnitude over 6, to the nearest number of its 8 bits; x over it goes to the
    nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6, ties to even codes."""
    x = x.unflatten(-1, (-1, 16))
    t = x.abs().amax(-1) / 6
    _, e = torch.frexp(t)
    step = torch.ldexp(torch.ones_like(t), e.clamp(min=-13) - 4)  # of the scale at this size; even steps on ties
    s = torch.clamp(torch.round(t / step) * step, max=61440.0)
    b = (s.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)
    y = torch.where(s[..., None] > 0, x / s[..., None], 0.0)
    a = y.abs()
    code = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, b


_CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _halves(byte):
    """The two 4-bit values of each byte, as fp32, side by side."""
    codes = torch.tensor(_CODES + [-v for v in _CODES], device=byte.device)
    return codes[torch.stack([byte & 15, byte >> 4], -1).flatten(-2).int()]


def _rows(s, name, index):
    """Rows of the pool as fp32, the index over (page, head, slot)."""
    kv = s["case"].get("kv", "e2m1")
    if kv == "bf16":
        return s[name][index].float()
    scale = s[name + "_scale"][index]
    if kv == "e4m3":
        return torch.ldexp(s[name].view(torch.uint8)[index].view(torch.float8_e4m3fn).float(), scale.int()[..., None] - 127)
    return (_halves(s[name][index]).unflatten(-1, (-1, 16)) * _level(scale)[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs

def _cache(c, lens, g, rng):
    """A pool of pages whose order is shuffled, and each sequence's table of them."""
    pages = [-(-n // c["page"]) for n in lens]
    total, width = max(1, sum(pages)) + 3, max(1, max(pages))
    order, at = rng.permutation(total), 0
    table = np.full((len(lens), width), -1, np.int32)
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p]
        at += p
    shape, kv = (total, c["kv_heads"], c["page"], c["dim"]), c.get("kv", "e2m1")
    s = {"table": torch.from_numpy(table).to(DEV), "k_scale": None, "v_scale": None}
    # a few channels of K are several times larger than the rest
    gain = torch.ones(c["dim"], device=DEV)
    gain[3::29] = 4.0
    for name, mul in (("k", gain), ("v", 0.5)):
        x = _randn(shape, g).mul_(mul)
        if kv == "bf16":
            s[name] = x.to(torch.bfloat16)
        else:
            s[name], s[name + "_scale"] = (_e4m3 if kv == "e4m3" else _e2m1)(x)
    return s


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    ints = lambda v: torch.from_numpy(np.asarray(v, np.int32)).to(DEV)  # noqa: E731
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if c["op"] == "table":  # another model's base
        s = {"base": float(10000 + 100 * rng.randint(0, 5000)), "table": torch.empty((c["positions"], c["dim"]), device=DEV)}
    elif c["op"] == "store":
        new, past = _spread(c["seqs"], 1, c["new"]), _spread(c["seqs"], 1, c["past"])
        rng.shuffle(new), rng.shuffle(past)
        lens = [a + b for a, b in zip(new, past)]
        s = _cache(c, lens, g, rng)
        t = sum(new)
        s["seq_ids"] = ints(np.repeat(np.arange(c["seqs"]), new))
        s["positions"] = ints(np.concatenate([np.arange(b, b + a) for a, b in zip(new, past)]))
        s["offsets"] = ints(np.concatenate([[0], np.cumsum(lens)]))
        a = np.arange(c["new"] + c["past"] + 1)[:, None] * 10000.0 ** (-np.arange(0, c["rotated"], 2) / c["rotated"])
        s["rope"] = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(DEV)
        s["q_out"] = torch.empty((t, c["q_heads"], c["dim"]), **bf16)
        for name, heads in (("q", c["q_heads"]), ("new_k", c["kv_heads"]), ("new_v", c["kv_heads"])):
            s[name] = _randn((t, heads, c["dim"]), g).to(torch.bfloat16)
        s["k_out"], s["v_out"] = (torch.empty((sum(lens), c["kv_heads"], c["dim"]), **bf16) for _ in "kv")
    else:
        if c["op"] == "token":
            lens = _ragged(c["seqs"], c["longest"])
            rng.shuffle(lens)
            s = {"lengths": ints(lens), "first": None, "prefix": None}
            rows = c["seqs"]
        else:
            new, lens, prefix, first = _prompts(c)
            s = {"lengths": ints(lens), "offsets": ints(np.concatenate([[0], np.cumsum(new)])),
                 "first": None if first is None else ints(first), "prefix": ints(prefix) if c["prefix"] else None}
            rows = sum(new)
        s.update(_cache(c, lens, g, rng))
        # the heads' slopes fall off as powers of two
        s["slopes"] = torch.exp2(-8 * torch.arange(1, c["q_heads"] + 1, device=DEV) / c["q_heads"]) if c["slopes"] else None
        s["q"] = _randn((rows, c["q_heads"], c["dim"]), g, 1.5).to(torch.bfloat16)
        s["out"] = torch.empty((rows, c["q_heads"], c["dim"]), **bf16)
        s["lse"] = torch.empty((rows, c["q_heads"]), dtype=torch.float32, device=DEV)
    s["case"] = c
    return s


# ---------------------------------------------------------------- plain forms

def _plain_table(s):
    c = s["case"]
    # angles of far positions need 64 bits
    f = s["base"] ** (-torch.arange(0, c["dim"], 2, dtype=torch.float64, device=DEV) / c["dim"])
    if c["factor"] != 1:
        keep = ((c["original"] * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    a = torch.arange(c["positions"], dtype=torch.float64, device=DEV)[:, None] * f
    return {"table": (torch.cat([a.cos(), a.sin()], 1) * c["amplitude"]).float()}


def _plain_store(s):
    c = s["case"]
    cos, sin = s["rope"][s["positions"].long()][:, None].chunk(2, -1)

    def rotated(x):
        x, rest = x.float().split([c["rotated"], c["dim"] - c["rotated"]], -1)
        a, b = (x[..., 0::2], x[..., 1::2]) if c["interleaved"] else x.chunk(2, -1)
        x = (a * cos - b * sin, b * cos + a * sin)
        return torch.cat([torch.stack(x, -1).flatten(-2) if c["interleaved"] else torch.cat(x, -1), rest], -1)

    at = s["positions"].long()
    pages = s["table"][s["seq_ids"].long(), at // c["page"]].long()
    for name, x in (("k", rotated(s["new_k"])), ("v", s["new_v"].float())):
        s[name][pages, :, at % c["page"]], s[name + "_scale"][pages, :, at % c["page"]] = _e2m1(x)
    t = torch.arange(s["k_out"].shape[0], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"], t, right=True) - 1
    at = (t - s["offsets"][seq]).long()
    index = (s["table"][seq, at // c["page"]].long(), slice(None), at % c["page"])
    return {"q": rotated(s["q"]).to(torch.bfloat16), "k": _rows(s, "k", index).to(torch.bfloat16), "v": _rows(s, "v", index).to(torch.bfloat16)}


def _plain_attention(s):
    """Every sequence padded to the longest; a single token is a prompt of one."""
    c = s["case"]
    lengths = s["lengths"].long()
    n, heads, kv_heads = c["seqs"], c["q_heads"], c["kv_heads"]
    if c["op"] == "token":
        offsets = torch.arange(n + 1, device=DEV)
        counts, most = (lengths > 0).long(), 1
    else:
        offsets = s["offsets"].long()
        counts, most = offsets.diff(), max(1, c["new"])
    row = torch.arange(most, device=DEV)
    live = row < counts[:, None]
    t = (offsets[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)  # token of (sequence, row)
    p = (lengths - counts)[:, None] + row                          # its position
    j = torch.arange(s["table"].shape[1] * c["page"], device=DEV)
    hi = p + 1 if s["prefix"] is None else torch.maximum(p + 1, s["prefix"][:, None])
    lo = torch.zeros_like(p) if s["first"] is None else s["first"].long()[t]
    lo = torch.maximum(lo, p + 1 - c["window"]) if c["window"] else lo
    seen = (j >= lo[..., None]) & (j < hi[..., None]) & live[..., None]
    index = (s["table"].clamp(min=0).long(),)
    k, v = (_rows(s, name, index).transpose(1, 2).reshape(n, kv_heads, 1, -1, c["dim"]) for name in "kv")
    v = torch.where(j[:, None] < lengths[:, None, None, None, None], v, 0.0)
    q = s["q"].float()[t].view(n, most, kv_heads, heads // kv_heads, c["dim"]).permute(0, 2, 3, 1, 4)
    x = q @ k.transpose(-1, -2) * (1 / math.sqrt(c["dim"]))
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    if c["slopes"]:
        x = x - s["slopes"].view(kv_heads, -1, 1, 1) * (p[..., None] - j).abs()[:, None, None]
    x = torch.where(seen[:, None, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    out = torch.where(total > 0, x @ v / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, most, heads, c["dim"])
    lse = (top + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(n, most, heads)
    if c["op"] == "token":
        return {"out": out[:, 0].to(torch.bfloat16), "lse": lse[:, 0]}
    at = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(offsets, at, right=True) - 1
    index = (seq, at - offsets[seq])
    return {"out": out[index].to(torch.bfloat16), "lse": lse[index]}


_PLAIN = {"table": _plain_table, "store": _plain_store, "token": _plain_attention, "prompt": _plain_attention}


# ---------------------------------------------------------------- one pass

def _own(s):
    from bit_delta_tenant_gb300 import bitdelta as bd

    c = s["case"]
    if c["op"] == "table":
        bd.bd_rotary_table(s["table"], s["base"], factor=c["factor"], original=c["original"], low=1.0, high=4.0,
                           amplitude=c["amplitude"])
        return {"table": s["table"]}
    cache = s.get("cache")
    if cache is None:  # a program keeps the cache's handle
        cache = s["cache"] = bd.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "store":
        bd.bd_kv_append_rotary(cache, s["q"], s["new_k"], s["new_v"], s["positions"], s["table"], s["rope"], s["q_out"],
                               seq_ids=s["seq_ids"], interleaved=c["interleaved"])
        bd.bd_kv_read(cache, s["table"], s["offsets"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    rule = dict(scale=1 / math.sqrt(c["dim"]), window=c["window"], cap=c["cap"], slopes=s["slopes"], first=s["first"], lse=s["lse"])
    token = c["op"] == "token"
    if "workspace" not in s:  # and one zero-filled workspace
        need = (bd.bd_attention_workspace_size(cache, c["seqs"], c["q_heads"]) if token
                else bd.bd_attention_prompt_workspace_size(cache, c["q_heads"]))
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    if token:
        bd.bd_attention_decode(cache, s["q"], s["table"], s["lengths"], s["out"], s["workspace"], **rule)
    else:
        bd.bd_attention_prompt(cache, s["q"], s["offsets"], s["table"], s["lengths"], s["out"], s["workspace"], prefix=s["prefix"],
                               **rule)
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


# ---------------------------------------------------------------- the definitions in 64 bits

def _host(t):
    return t.double().cpu().numpy()


def _exact_table(s):
    c = s["case"]
    i = np.arange(c["dim"] // 2)
    turns = np.exp(-2 * i / c["dim"] * math.log(s["base"])) / (2 * math.pi)  # per position
    if c["factor"] != 1:
        mix = np.clip((c["original"] * turns - 1.0) / (4.0 - 1.0), 0, 1)
        turns = mix * turns + (1 - mix) * turns / c["factor"]
    z = c["amplitude"] * np.exp(2j * math.pi * np.remainder(np.outer(np.arange(c["positions"]), turns), 1.0))
    return {"table": np.concatenate([z.real, z.imag], 1)}


def _exact_scale(top):
    """Of maxima of 16 values: nearest to a sixth of each, among numbers of 4 significant bits from 2^-14 on, of steps of 2^-17 below."""
    t = top / 6
    unit = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(t, 1e-300))), -14) - 3)
    return np.minimum(np.round(t / unit) * unit, 61440.0)


def _exact_four(x):
    """What rows x stand for once held in 4 bits."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = _exact_scale(np.abs(g).max(-1))[..., None]
    y = np.divide(np.abs(g), s, out=np.zeros_like(g), where=s > 0)
    code = np.searchsorted([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], y)  # ties go down
    tie = np.isin(y, [0.75, 1.75, 3.5])                                 # up to an even code here
    return (np.sign(g) * np.array(_CODES)[code + tie] * s).reshape(x.shape)


def _stored(s, name):
    """The pool's values in 64 bits, [page, head, slot, dim] on the device."""
    kv = s["case"].get("kv", "e2m1")
    if kv == "bf16":
        return s[name].double()
    b = s[name + "_scale"].double()
    if kv == "e4m3":
        return s[name].double() * torch.exp2(b - 127)[..., None]
    x = s[name].int()
    code = torch.stack([x % 16, x // 16], -1).flatten(-2)
    e, m = (code % 8 // 2).double(), (code % 2).double()
    x = torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2) * torch.where(code >= 8, -1.0, 1.0)
    e, m = torch.div(b, 8, rounding_mode="floor"), b % 8
    scale = torch.where(e > 0, torch.exp2(e - 15) * (1 + m / 8), m * 2.0 ** -17)
    return x * scale.repeat_interleave(16, -1)


def _exact_store(s):
    c = s["case"]
    pos, seq, table = (s[k].cpu().numpy().astype(np.int64) for k in ("positions", "seq_ids", "table"))
    d = c["rotated"] // 2
    angle = _host(s["rope"])[pos]
    turn = (angle[:, :d] + 1j * angle[:, d:])[:, None]
    pairs = (np.arange(0, 2 * d, 2), np.arange(1, 2 * d, 2)) if c["interleaved"] else (np.arange(d), np.arange(d, 2 * d))

    def rotated(x):
        x = _host(x)
        z = (x[..., pairs[0]] + 1j * x[..., pairs[1]]) * turn
        x[..., pairs[0]], x[..., pairs[1]] = z.real, z.imag
        return x

    ends = s["offsets"].cpu().numpy().astype(np.int64)
    out = {"q": rotated(s["q"])}
    for name, x in (("k", rotated(s["new_k"])), ("v", _host(s["new_v"]))):
        pool = _stored(s, name).cpu().numpy()
        rows = [pool[table[i, np.arange(b - a) // c["page"]], :, np.arange(b - a) % c["page"]] for i, (a, b) in enumerate(zip(ends, ends[1:]))]
        out[name] = np.concatenate(rows)
        out[name][ends[seq] + pos] = _exact_four(x)
    return out


def _exact_attention(s):
    c = s["case"]
    heads, dim = c["q_heads"], c["dim"]
    rows, group = s["q"].shape[0], heads // c["kv_heads"]
    out = torch.zeros((rows, heads, dim), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, heads), -torch.inf, dtype=torch.float64, device=DEV)
    token = c["op"] == "token"
    ends = list(range(rows + 1)) if token else s["offsets"].tolist()
    for i, length in enumerate(s["lengths"].tolist()):
        a, n = ends[i], ends[i + 1] - ends[i]
        if not length or not n:
            continue
        j = torch.arange(length, device=DEV)
        page, slot = s["table"][i].long().index_select(0, j.div(c["page"], rounding_mode="floor")), j % c["page"]
        p = torch.arange(length - n, length, device=DEV)[:, None]
        hidden = j > p
        if s["prefix"] is not None:
            hidden &= j >= s["prefix"][i]
        if c["window"]:
            hidden |= p - j >= c["window"]
        if s["first"] is not None:
            hidden |= j < s["first"][a:a + n, None]
        for h in range(c["kv_heads"]):
            part = {}
            for name in "kv":
                one = {"case": c, name: s[name][page, h, slot] if c["kv"] != "e4m3" else s[name].view(torch.uint8)[page, h, slot].view(torch.float8_e4m3fn)}
                if c["kv"] != "bf16":
                    one[name + "_scale"] = s[name + "_scale"][page, h, slot]
                part[name] = _stored(one, name)
            for head in range(h * group, (h + 1) * group):
                x = s["q"][a:a + n, head].double() @ part["k"].T / math.sqrt(dim)
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["slopes"]:
                    x = x - s["slopes"][head].double() * (p - j).abs()
                x = x.masked_fill(hidden, -torch.inf)
                lse[a:a + n, head] = torch.logsumexp(x, -1)
                out[a:a + n, head] = torch.softmax(x, -1).nan_to_num(0.0) @ part["v"]
    return {"out": out, "lse": lse}


def exact(c, seed):
    s = prepare(c, seed)
    return {"table": _exact_table, "store": _exact_store, "token": _exact_attention, "prompt": _exact_attention}[c["op"]](s)
