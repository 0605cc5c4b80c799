"""Measured cases of rotary positions and latent attention.

Latent attention keeps one row of 576 values a token for all heads: a latent
vector c of 512, which stands for keys and values, and 64 rotated columns k.

``rope``    Rotary positions of some columns of each head of q and k: pairs
            (i, i + R/2), or (2i, 2i + 1) where interleaved, turn by pos * f_i;
            the inverse turns back, which is also the gradient.
``write``   New tokens' rows [c | k] into the paged cache: c as it is or
            normalised by its root mean square and a weight, k rotated.
``cache``   Absorbed form over the paged cache: softmax(scale q [c | k]^T) c for
            packed queries, every head over the same rows.
``sparse``  The same over lists of rows: O and LSE of top-k sparse attention, as
            its backward takes them.
``prompt``  Expanded form: every head has keys of its own in 128 columns beside
            the 64 shared rotated ones, and values of 128; causal prompts, packed
            ones among them, or chunks against more keys than queries.

``run`` computes them in elementary torch operations in 32 bits (angles in 64),
or, with ``own``, calls this package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
ROW, LAT, ROT = 576, 512, 64  # a latent row, its latent vector, its rotated columns
NOPE, DV = 128, 128           # the expanded form's own key columns and values a head


def listed():
    return [
        # one decode step's queries and keys, far into long contexts: latency
        dict(op="rope", name="rope_decode", dtype="bf16", b=32, s=1, far=131071, hq=32, hk=8, dq=128, dk=128, rot=128,
             sq=0, sk=0, inter=False, inverse=False, base=10000.0, kind="parts", factor=8.0, length=16384, mix=1),
        # queries and keys of a 16384-token sequence before attention, positions stretched
        dict(op="rope", name="rope_prompt", dtype="bf16", b=1, s=16384, far=0, hq=32, hk=4, dq=128, dk=128, rot=128,
             sq=0, sk=0, inter=False, inverse=False, base=10000.0, kind="linear", factor=4.0, length=4096, mix=2),
        # the gradients of absorbed queries and latent rows, turned back: 64 columns of 576
        dict(op="rope", name="rope_latent_gradient", dtype="bf16", b=1, s=4096, far=0, hq=64, hk=1, dq=ROW, dk=ROW,
             rot=ROT, sq=LAT, sk=LAT, inter=True, inverse=True, base=10000.0, kind="none", factor=1.0, length=4096, mix=3),
        # one token of every request of a server, normalised and rotated as it is written
        dict(op="write", name="latent_write_decode", dtype="bf16", n=128, ctx=8191, new=1, page=64, norm=True, rope=True,
             inter=True, mix=4),
        # prompts of all lengths written in one go
        dict(op="write", name="latent_write_prompts", dtype="f16", n=13, ctx=200, new=4096, page=32, norm=True, rope=True,
             inter=False, mix=5),
        # one user, a short conversation, few heads: the latency of the smallest call
        dict(op="cache", name="latent_one_short", dtype="bf16", n=1, ctx=384, new=1, h=16, page=16, causal=True, mix=6),
        # the decode step of a loaded server
        dict(op="cache", name="latent_decode", dtype="bf16", n=64, ctx=8191, new=1, h=64, page=64, causal=True, mix=7),
        # drafted tokens of few requests with long contexts, all heads on one GPU
        dict(op="cache", name="latent_drafts_long", dtype="f16", n=5, ctx=65535, new=3, h=128, page=32, causal=True, mix=8),
        # lists with holes and empty rows, few tokens
        dict(op="sparse", name="sparse_small", dtype="f16", b=1, s=140, skv=140, h=32, g=1, topk=130, holes=0.3, mix=9),
        # the forward of a top-k training step: 2048 of 4096 rows a token
        dict(op="sparse", name="sparse_train", dtype="bf16", b=1, s=4096, skv=4096, h=64, g=1, topk=2048, holes=0.0,
             mix=10),
        # a chunk of a prompt against what came before it
        dict(op="prompt", name="latent_prompt_chunk", dtype="bf16", b=1, s=2048, sk=8192, h=64, packed=0, causal=True,
             mix=11),
        # prompts of unequal lengths packed into one call
        dict(op="prompt", name="latent_prompts_packed", dtype="f16", b=1, s=16384, sk=16384, h=16, packed=4, causal=True,
             mix=12),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = {}
    for c in listed():
        w = work(c)
        for k in w:
            most[c["op"], k] = max(most.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["rope", "write", "cache", "cache", "sparse", "prompt"])
        c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), mix=rng.randrange(100, 1 << 20))
        if op == "rope":
            rot = rng.choice([16, 32, 64, 96, 128])
            sq, sk = 8 * rng.randrange(0, 5), 8 * rng.randrange(0, 5)
            kind = rng.choice(["none", "linear", "base", "parts"])
            c.update(b=log(1, 64), s=log(1, 16384), far=rng.choice([0, log(1, 1000000)]), hq=rng.choice([1, 3, 16, 32, 64]),
                     hk=rng.choice([0, 1, 2, 5, 8]), dq=sq + rot + 8 * rng.randrange(0, 5), dk=sk + rot + 8 * rng.randrange(0, 5),
                     rot=rot, sq=sq, sk=sk, inter=rng.random() < 0.5, inverse=rng.random() < 0.5,
                     base=rng.choice([10000.0, 500000.0]), kind=kind, factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 32.0]),
                     length=rng.choice([2048, 8192]))
        elif op == "write":
            norm = rng.random() < 0.7
            c.update(n=log(1, 300), ctx=log(1, 16384), new=rng.choice([1, log(2, 16), log(2, 4096)]),
                     page=rng.choice([16, 32, 64, 128]), norm=norm, rope=rng.random() < 0.8, inter=rng.random() < 0.5)
            if sum(_lens(c)[2]) > 1 << 19:  # the cache that is compared
                continue
        elif op == "cache":
            c.update(n=log(1, 200), ctx=log(1, 100000), new=rng.choice([1, 1, log(2, 8), log(2, 300)]),
                     h=rng.choice([1, 8, 16, 20, 32, 64, 96, 128]), page=rng.choice([16, 32, 64, 128]),
                     causal=rng.random() < 0.8)
            if sum(_lens(c)[2]) > 1 << 19 or c["n"] * (c["ctx"] + c["new"]) > 1 << 19:  # the padded plain form's keys
                continue
            if c["n"] * c["new"] * c["h"] * (c["ctx"] + c["new"]) > 1 << 30:  # and its scores
                continue
        elif op == "sparse":
            g = rng.choice([1, 1, 2])
            s = log(1, 4096)
            c.update(b=rng.choice([1, 1, 2]), s=s, skv=rng.choice([s, log(1, 8192)]), h=g * rng.choice([1, 8, 16, 24, 32, 64]),
                     g=g, topk=log(1, 2048), holes=rng.choice([0.0, 0.3]))
            if c["b"] * s * g * max(c["topk"], c["skv"] // 4) > 1 << 23:  # the plain form's rows, and what draws the lists
                continue
        else:
            packed = rng.choice([0, 0, log(2, 40)])
            s = log(1, 16384)
            b = 1 if packed else rng.choice([1, 1, 2, 3])
            causal = rng.random() < 0.8
            c.update(b=b, s=s, sk=s if packed else rng.choice([s, s + log(1, 8192), log(1, 16384)]),
                     h=rng.choice([1, 4, 16, 20, 64, 128]), packed=packed, causal=causal)
            if c["b"] * c["h"] * c["s"] * c["sk"] > 1 << 32:  # the plain form's scores
                continue
        w = work(c)
        if w["bytes"] <= most[op, "bytes"] and w["flops"] <= most[op, "flops"]:
            return c


def _lens(c):
    """Cached tokens before the call, new tokens, and key lengths, by the case alone."""
    r = random.Random(c["mix"])
    n = c["n"]
    ctx = [c["ctx"]] + [r.randint(0, c["ctx"]) for _ in range(n - 1)]
    new = [c["new"]] + [r.randint(0 if c["new"] > 1 else 1, c["new"]) for _ in range(n - 1)]
    return ctx, new, [a + b for a, b in zip(ctx, new)]


def _bounds(c):
    """Bounds of packed sequences."""
    if c["s"] == 16384 and c["packed"] == 4:
        return [0, 3000, 8000, 9537, 16384]
    r = random.Random(c["mix"])
    return [0] + sorted(r.randint(0, c["s"]) for _ in range(c["packed"] - 1)) + [c["s"]]


def _listed_rows(c):
    """How many slots of all index lists hold a row (holes as they are expected), and rows that some list may hold."""
    t = np.arange(c["s"], dtype=np.int64) + max(0, c["skv"] - c["s"])
    seen = np.minimum(np.minimum(t + 1, c["skv"]), c["topk"]).sum()
    return c["b"] * c["g"] * int(seen * (1 - c["holes"])), c["b"] * c["g"] * c["skv"]


def _pairs(c):
    """Visible (query, key) pairs of the expanded form."""
    if c["packed"]:
        cu = _bounds(c)
        n = [b - a for a, b in zip(cu[:-1], cu[1:])]
        return sum(x * (x + 1) // 2 if c["causal"] else x * x for x in n)
    if not c["causal"]:
        return c["b"] * c["s"] * c["sk"]
    last = np.arange(c["s"], dtype=np.int64) + c["sk"] - c["s"] + 1
    return c["b"] * int(np.clip(last, 0, c["sk"]).sum())


def work(c):
    op = c["op"]
    if op == "rope":  # the turned columns in and out, a position a token
        n = c["b"] * c["s"]
        whole = c["dq"] != ROW  # (elsewhere the other columns stay where they are: the call is in place)
        cols = c["hq"] * (c["dq"] if whole else c["rot"]) + c["hk"] * (c["dk"] if whole else c["rot"])
        return {"bytes": n * (4 * cols + 4), "flops": n * (c["hq"] + c["hk"]) * c["rot"] * 3}
    if op == "write":
        T = sum(_lens(c)[1])
        return {"bytes": T * (4 * ROW + 8), "flops": T * (4 * LAT + 3 * ROT)}
    if op == "cache":
        ctx, new, kv = _lens(c)
        pairs = sum(m * L - (m * (m - 1) // 2 if c["causal"] else 0) for m, L in zip(new, kv))
        T, keys = sum(new), sum(L for m, L in zip(new, kv) if m)
        return {"bytes": keys * ROW * 2 + 4 * (keys // c["page"]) + T * c["h"] * (2 * (ROW + LAT) + 4),
                "flops": 2 * (ROW + LAT) * c["h"] * pairs}
    if op == "sparse":
        slots, rows = _listed_rows(c)
        T = c["b"] * c["s"]
        return {"bytes": 2 * rows * ROW + 4 * T * c["g"] * c["topk"] + T * c["h"] * (2 * (ROW + LAT) + 4),
                "flops": 2 * (ROW + LAT) * (c["h"] // c["g"]) * slots}
    T, K = c["b"] * c["s"], c["b"] * c["sk"]
    return {"bytes": T * c["h"] * (2 * (NOPE + ROT + DV) + 4) + K * (2 * c["h"] * (NOPE + DV) + 2 * ROT),
            "flops": 2 * (NOPE + ROT + DV) * c["h"] * _pairs(c)}


# ------------------------------------------------------------------ inputs


def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt * 7919) & 0x7FFFFFFF)


def _randn(shape, c, seed, salt):
    return torch.randn(shape, generator=_gen(seed, salt), device="cuda").to(DT[c["dtype"]])


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _pages(c, seed):
    """Block table of every request's pages (-1 behind them), in shuffled blocks."""
    kv, p = _lens(c)[2], c["page"]
    need = [(x + p - 1) // p for x in kv]
    nb = sum(need) + 7
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(nb).astype(np.int32)
    table = np.full((c["n"], max(need)), -1, np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = order[at:at + m]
        at += m
    return table, nb


def _prepare_rope(c, seed):
    s = {"q": _randn((c["b"], c["s"], c["hq"], c["dq"]), c, seed, 1)}
    if c["hk"]:
        s["k"] = _randn((c["b"], c["s"], c["hk"], c["dk"]), c, seed, 2)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    first = r.randint(0, c["far"] + 1, size=(c["b"], 1))  # where each row of the batch begins
    s["pos"] = _i32(first + np.arange(c["s"])[None, :])
    return s


def _prepare_write(c, seed):
    ctx, new, kv = _lens(c)
    p, T = c["page"], sum(new)
    table, nb = _pages(c, seed)
    pos = [np.arange(a, a + m) for a, m in zip(ctx, new)]
    slots = [table[r, x // p] * p + x % p for r, x in enumerate(pos)]
    s = dict(kv=_randn((1, T, ROW), c, seed, 1), cache=_randn((nb, p, ROW), c, seed, 2), slots=_i32(np.concatenate(slots)),
             pos=_i32(np.concatenate(pos)))
    if c["norm"]:
        s["weight"] = (1 + 0.2 * torch.randn(LAT, generator=_gen(seed, 3), device="cuda")).to(DT[c["dtype"]])
    return s


def _prepare_cache(c, seed):
    ctx, new, kv = _lens(c)
    table, nb = _pages(c, seed)
    return dict(q=_randn((1, sum(new), c["h"], ROW), c, seed, 1), cache=_randn((nb, c["page"], ROW), c, seed, 2),
                table=_i32(table), kv=_i32(kv), cu=_i32(np.concatenate([[0], np.cumsum(new)])), m=max(new), L=max(kv),
                scale=(NOPE + ROT) ** -0.5)


def _prepare_sparse(c, seed):
    B, S, K, G, n = c["b"], c["s"], c["skv"], c["g"], c["topk"]
    t = torch.arange(S, device="cuda") + max(0, K - S)  # the last token sees the last row
    key = torch.rand((B, S, G, K), generator=_gen(seed, 3), device="cuda")
    key.masked_fill_(torch.arange(K, device="cuda")[None, None, None, :] > t[None, :, None, None], -1.0)
    top, idx = key.topk(min(n, K), dim=-1)
    idx = torch.where(top >= 0, idx, torch.full_like(idx, K)).sort(-1).values
    idx = torch.where(idx < K, idx, torch.full_like(idx, -1))
    if c["holes"]:
        gone = torch.rand(idx.shape, generator=_gen(seed, 4), device="cuda") < c["holes"]
        gone |= torch.rand((B, S, G, 1), generator=_gen(seed, 5), device="cuda") < 0.05  # lists without a row
        idx = idx.masked_fill(gone, -1)
    idx = torch.nn.functional.pad(idx, (0, n - idx.shape[-1]), value=-1).int().contiguous()
    return dict(q=_randn((B, S, c["h"], ROW), c, seed, 1), rows=_randn((B, K, G, ROW), c, seed, 2), idx=idx,
                scale=ROW ** -0.5)


def _prepare_prompt(c, seed):
    B, S, K, H = c["b"], c["s"], c["sk"], c["h"]
    # a projection of the latent vectors makes each head's keys and values side by side
    up = _randn((B, K, H, NOPE + DV), c, seed, 2)
    s = dict(q=_randn((B, S, H, NOPE + ROT), c, seed, 1), k=up[..., :NOPE], v=up[..., NOPE:],
             kr=_randn((B, K, ROT), c, seed, 3), scale=(NOPE + ROT) ** -0.5)
    if c["packed"]:
        s["cu"] = _i32(_bounds(c))
    return s


def prepare(c, seed):
    s = {"rope": _prepare_rope, "write": _prepare_write, "cache": _prepare_cache, "sparse": _prepare_sparse,
         "prompt": _prepare_prompt}[c["op"]](c, seed)
    s["c"] = c
    if own and (c["op"] == "rope" or c["op"] == "write" and c["rope"]):
        import attention_backward_gb300 as ab

        # the frequencies, which a program makes once
        if c["op"] == "rope":
            s["turns"] = ab.rope_table(c["rot"], c["base"], scaling=c["kind"], factor=c["factor"], original_length=c["length"])
        else:
            s["turns"] = ab.rope_table(ROT)
    return s


# ------------------------------------------------------------------ the plain forms


def _frequencies(c, device):
    """f_i = base^(-2i/R) in f64, stretched: ``linear`` all of them by the factor,
    ``base`` by a larger base, ``parts`` those that turn fewer than once in
    ``length`` positions by the factor, those that turn more than 32 times not at all,
    and in between by a ramp over i; and the factor of the result."""
    R, base, f = c["rot"], c["base"], c["factor"]
    i = torch.arange(R // 2, dtype=torch.float64, device=device)
    if c["kind"] == "base":
        base = base * f ** (R / (R - 2))
    w = torch.pow(torch.tensor(base, dtype=torch.float64, device=device), -2 * i / R)
    if c["kind"] == "linear":
        return w / f, 1.0
    if c["kind"] != "parts":
        return w, 1.0

    def at(turns):  # the i whose pair turns so often
        return R * math.log(c["length"] / (turns * 2 * math.pi)) / (2 * math.log(c["base"]))

    lo, hi = max(0, math.floor(at(32))), min(R // 2 - 1, math.ceil(at(1)))
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return w * (1 - ramp) + w / f * ramp, 0.1 * math.log(f) + 1


def _turned(x, start, rot, cos, sin, inter):
    """x in 32 bits with its pairs turned (cos, sin [..., R/2])."""
    y = x.float()
    z = y[..., start:start + rot]
    if inter:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y[..., :start], z, y[..., start + rot:]], -1)


def _plain_rope(s):
    c = s["c"]
    w, scale = _frequencies(c, s["q"].device)
    t = s["pos"].double()[:, :, None, None] * w
    cos, sin = (t.cos() * scale).float(), (t.sin() * (-scale if c["inverse"] else scale)).float()
    out = []
    for name, start in (("q", c["sq"]), ("k", c["sk"])):
        if name in s:
            y = _turned(s[name], start, c["rot"], cos, sin, c["inter"]).to(s[name].dtype)
            out.append(s[name].copy_(y) if c["dq"] == ROW else y)
    return out


def _plain_write(s):
    c, x = s["c"], s["kv"][0].float()
    lat, rot = x[:, :LAT], x[:, LAT:]
    if c["norm"]:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    if c["rope"]:
        w = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device),
                      -torch.arange(0, ROT, 2, dtype=torch.float64, device=x.device) / ROT)
        t = s["pos"].double()[:, None] * w
        rot = _turned(rot, 0, ROT, t.cos().float(), t.sin().float(), c["inter"])
    s["cache"].view(-1, ROW)[s["slots"].long()] = torch.cat([lat, rot], -1).to(s["cache"].dtype)
    return [s["cache"]]


def _softmax_parts(x):
    """exp(x - top), its sum and top along the last axis; rows of -inf give zeros."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x.sub_(top).exp_()
    return x, x.sum(-1, keepdim=True), top


def _divided(o, total):
    return torch.where(total > 0, o / total, torch.zeros_like(o))


def _plain_cache(s):
    c, q = s["c"], s["q"][0]
    T, H, _ = q.shape
    n, m, p = c["n"], s["m"], c["page"]
    kv, cu = s["kv"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)
    qp = q[rows].float().view(n, m * H, ROW)
    k = s["cache"][s["table"].long().clamp(min=0)].float().view(n, -1, ROW)
    j = torch.arange(k.shape[1], device=q.device)
    see = j[None, None, :] < kv[:, None, None]
    if c["causal"]:
        see = see & (j[None, None, :] <= ((kv - new)[:, None] + i[None, :])[:, :, None])
    x = torch.matmul(qp, k.transpose(1, 2)).mul_(s["scale"]).view(n, m, H, -1)
    x.masked_fill_(~see[:, :, None, :], -math.inf)
    x, total, top = _softmax_parts(x)
    o = torch.matmul(x.view(n, m * H, -1), k[..., :LAT]).view(n, m, H, LAT)
    o = _divided(o, total)
    lse = (total.log() + top)[..., 0]
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    at = t - cu[r]
    return [o[r, at][None].to(q.dtype), lse[r, at].t().contiguous()[None]]


def _plain_sparse(s):
    c, idx = s["c"], s["idx"].long()
    B, S, G, n = idx.shape
    see = (idx >= 0) & (idx < c["skv"])
    b = torch.arange(B, device=idx.device)[:, None, None, None]
    g = torch.arange(G, device=idx.device)[None, None, :, None]
    k = s["rows"][b, idx.clamp(0, c["skv"] - 1), g].float()  # [B, S, G, n, 576]
    q = s["q"].float().view(B, S, G, c["h"] // G, ROW)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    x.masked_fill_(~see[:, :, :, None, :], -math.inf)
    x, total, top = _softmax_parts(x)
    o = _divided(torch.matmul(x, k[..., :LAT]), total).view(B, S, c["h"], LAT)
    lse = (total.log() + top).view(B, S, c["h"]).transpose(1, 2).contiguous()
    return [o.to(s["q"].dtype), lse]


def _plain_prompt(s):
    c = s["c"]
    q = s["q"].float().transpose(1, 2)  # [B, H, S, 192]
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    kr = s["kr"].float()[:, None]
    x = torch.matmul(q[..., :NOPE], k.transpose(2, 3))
    x += torch.matmul(q[..., NOPE:], kr.transpose(2, 3))
    x.mul_(s["scale"])
    i = torch.arange(c["s"], device=x.device)[:, None]
    j = torch.arange(c["sk"], device=x.device)[None, :]
    see = (j <= i + c["sk"] - c["s"]) if c["causal"] else torch.ones_like(i + j, dtype=torch.bool)
    if c["packed"]:
        cu = s["cu"].long()
        see = see & (torch.searchsorted(cu, i, right=True) == torch.searchsorted(cu, j, right=True))
    x.masked_fill_(~see, -math.inf)
    x, total, top = _softmax_parts(x)
    o = _divided(torch.matmul(x, v), total)
    return [o.transpose(1, 2).contiguous().to(s["q"].dtype), (total.log() + top)[..., 0]]


def _own(s):
    import attention_backward_gb300 as ab

    c = s["c"]
    if c["op"] == "rope":
        out = (s["q"], s.get("k")) if c["dq"] == ROW else None
        q, k = ab.rope(s["q"], s["pos"], s["turns"], k=s.get("k"), interleaved=c["inter"], start=c["sq"], k_start=c["sk"],
                       inverse=c["inverse"], out=out)
        return [q] if k is None else [q, k]
    if c["op"] == "write":
        ab.latent_cache_write(s["kv"], s["slots"], s["cache"], norm_weight=s.get("weight"), norm_eps=1e-6,
                              positions=s["pos"] if c["rope"] else None, table=s.get("turns"), interleaved=c["inter"])
        return [s["cache"]]
    if c["op"] == "cache":
        return list(ab.forward_latent_cache(s["q"], s["cache"], s["table"], s["cu"], s["kv"], s["scale"], causal=c["causal"]))
    if c["op"] == "sparse":
        return list(ab.sparse_forward(s["q"], s["rows"], s["idx"], s["scale"], LAT))
    return list(ab.forward_latent(s["q"], s["k"], s["kr"], s["v"], s["scale"], causal=c["causal"], cu_seqlens=s.get("cu")))


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "write": _plain_write, "cache": _plain_cache, "sparse": _plain_sparse,
            "prompt": _plain_prompt}[s["c"]["op"]](s)


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _rotations(pos, R, base, kind="none", f=1.0, length=0):
    """e^(i pos f_i) times the result's factor, complex128 [..., R/2]."""
    scale, out = 1.0, []
    for i in range(R // 2):
        w = base ** (-2 * i / R)
        if kind == "linear":
            w /= f
        elif kind == "base":
            w = (base * f ** (R / (R - 2))) ** (-2 * i / R)
        elif kind == "parts":
            first = max(0, math.floor(R / 2 * math.log(length / (64 * math.pi), base)))
            last = min(R // 2 - 1, math.ceil(R / 2 * math.log(length / (2 * math.pi), base)))
            part = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            w *= 1 - part + part / f
            scale = 1 + math.log(f) / 10
        out.append(w)
    t = pos.double()[..., None] * torch.tensor(out, dtype=torch.float64, device=pos.device)
    return torch.polar(torch.full_like(t, scale), t)


def _exact_turn(x, start, R, z, inter):
    y = x.double().clone()
    part = y[..., start:start + R].clone()
    if inter:
        turned = torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (R // 2, 2)).contiguous()) * z)
        y[..., start:start + R] = turned.flatten(-2)
    else:
        turned = torch.complex(part[..., :R // 2].contiguous(), part[..., R // 2:].contiguous()) * z
        y[..., start:start + R] = torch.cat([turned.real, turned.imag], -1)
    return y


def _exact_rows(q, k, scale, see):
    """O and LSE of rows q over rows k [.., 576]: see True where a key counts."""
    x = (q @ k.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.where(torch.isinf(lse)[..., None], torch.zeros_like(x), torch.exp(x - lse[..., None]))
    return p @ k[..., :LAT], lse


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        z = _rotations(s["pos"], c["rot"], c["base"], c["kind"], c["factor"], c["length"])[:, :, None]
        z = z.conj() if c["inverse"] else z
        return [_exact_turn(s[x], c[at], c["rot"], z, c["inter"]) for x, at in (("q", "sq"), ("k", "sk")) if x in s]
    if c["op"] == "write":
        x = s["kv"][0].double()
        if c["rope"]:
            x = _exact_turn(x, LAT, ROT, _rotations(s["pos"], ROT, 10000.0), c["inter"])
        if c["norm"]:
            r = torch.sqrt((x[:, :LAT] ** 2).sum(1, keepdim=True) / LAT + 1e-6)
            x[:, :LAT] = x[:, :LAT] / r * s["weight"].double()
        cache = s["cache"].double()
        p = c["page"]
        for t, slot in enumerate(s["slots"].tolist()):
            cache[slot // p, slot % p] = x[t]
        return [cache]
    if c["op"] == "cache":
        T, H, p = s["q"].shape[1], c["h"], c["page"]
        o = torch.zeros(1, T, H, LAT, dtype=torch.float64, device="cuda")
        lse = torch.full((1, H, T), -math.inf, dtype=torch.float64, device="cuda")
        cu, table = s["cu"].tolist(), s["table"].tolist()
        for r, L in enumerate(s["kv"].tolist()):
            m = cu[r + 1] - cu[r]
            if m == 0 or L == 0:
                continue
            blocks = torch.tensor(table[r][:(L + p - 1) // p], device="cuda")
            k = s["cache"][blocks].double().reshape(-1, ROW)[:L]
            far = torch.arange(L, device="cuda")[None, :] - (torch.arange(m, device="cuda")[:, None] + L - m)
            see = far <= 0 if c["causal"] else far < L
            for h in range(H):
                o[0, cu[r]:cu[r + 1], h], lse[0, h, cu[r]:cu[r + 1]] = _exact_rows(s["q"][0, cu[r]:cu[r + 1], h].double(), k,
                                                                                  s["scale"], see)
        return [o, lse]
    if c["op"] == "sparse":
        B, S, G, n = s["idx"].shape
        e = c["h"] // G
        o = torch.zeros(B, S, c["h"], LAT, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, c["h"], S, dtype=torch.float64, device="cuda")
        for b in range(B):
            for g in range(G):
                rows, heads = s["rows"][b, :, g].double(), slice(g * e, (g + 1) * e)
                for t in range(0, S, 128):
                    idx = s["idx"][b, t:t + 128, g].long()
                    see = (idx >= 0) & (idx < c["skv"])
                    k = rows[torch.where(see, idx, torch.zeros_like(idx))]
                    o[b, t:t + 128, heads], z = _exact_rows(s["q"][b, t:t + 128, heads].double(), k, s["scale"], see[:, None])
                    lse[b, heads, t:t + 128] = z.t()
        return [o, lse]
    B, S, K, H = c["b"], c["s"], c["sk"], c["h"]
    o = torch.zeros(B, S, H, DV, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, S), -math.inf, dtype=torch.float64, device="cuda")
    cu = _bounds(c) if c["packed"] else [0, S]
    for b in range(B):
        for h in range(H):
            k = torch.cat([s["k"][b, :, h], s["kr"][b]], -1).double()
            v, q = s["v"][b, :, h].double(), s["q"][b, :, h].double()
            for a, e in zip(cu[:-1], cu[1:]):
                keys = slice(a, e) if c["packed"] else slice(0, K)
                for r in range(a, e, 4096):
                    rows = slice(r, min(e, r + 4096))
                    x = q[rows] @ k[keys].T * s["scale"]
                    if c["causal"]:
                        i = torch.arange(rows.start, rows.stop, device="cuda")[:, None] + (0 if c["packed"] else K - S)
                        x.masked_fill_(torch.arange(keys.start, keys.stop, device="cuda")[None, :] > i, -math.inf)
                    z = torch.logsumexp(x, -1)
                    p = torch.where(torch.isinf(z)[:, None], torch.zeros_like(x), torch.exp(x - z[:, None]))
                    o[b, rows, h], lse[b, h, rows] = p @ v[keys], z
    return [o, lse]
