"""Measured cases of the serving operators over a paged 8-bit key/value cache.

Three operators, used one after another in every step of a server:

``tables``  Block tables and slot maps from request lengths.  Request n holds
            ctx[n] tokens and gets new[n] more; page j of a request covers its
            positions [j P, (j + 1) P).  The pages it lacks are taken from the
            free list in request order, and each new token gets its slot
            (block * P + offset), its position, and its request's range of
            packed rows.
``write``   New keys and values appended to the cache as e4m3 with one scale
            for each page and KV head: the least power of two s with
            max|x| <= 448 s over the page's tokens.  A page that already holds
            tokens keeps its scale unless the new tokens need a larger one; its
            older values are then rounded again at the new scale.
``attend``  softmax(scale q k^T) v over the cached keys, packed queries of
            unequal counts, grouped heads, causal (the last query sees the last
            key), sliding window or unmasked; O in the query's type and the
            natural-log LSE in f32.

``run`` computes them in elementary torch operations in 32 bits, or, with
``own``, calls this package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100  # scales are at least 2^-100
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _case(op, name=None, *, n, ctx, new=1, dtype="bf16", hq=32, hkv=8, d=128, page=64, causal=True, window=-1, mix=1):
    c = dict(op=op, n=n, ctx=ctx, new=new, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, causal=causal, window=window,
             mix=mix)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step of a full server: every request one token further, small pages
        _case("tables", "tables_decode", n=256, ctx=8192, new=1, page=16, mix=11),
        # admission of many prompts at once, some of them continuing
        _case("tables", "tables_prompts", n=97, ctx=16384, new=2048, page=64, mix=12),
        # the same decode step's keys and values: one token to each request's last page
        _case("write", "write_decode", n=256, ctx=512, new=1, dtype="bf16", hkv=8, d=128, page=16, mix=13),
        # prompts written in one go, starting inside pages as well as at their start
        _case("write", "write_prompts", n=13, ctx=200, new=4096, dtype="f16", hkv=4, d=128, page=64, mix=14),
        # short prompts at head dim 64
        _case("write", "write_prompts_d64", n=37, ctx=50, new=257, dtype="bf16", hkv=8, d=64, page=16, mix=15),
        # one user, a short conversation: the latency of the smallest call
        _case("attend", "attend_one_short", n=1, ctx=384, new=1, dtype="bf16", hq=32, hkv=8, d=128, page=16, mix=16),
        # the decode step of a loaded server, lengths of all kinds
        _case("attend", "attend_decode", n=64, ctx=8191, new=1, dtype="bf16", hq=32, hkv=8, d=128, page=64, mix=17),
        # few requests with very long contexts: few rows over a long axis
        _case("attend", "attend_decode_long", n=3, ctx=131071, new=1, dtype="f16", hq=32, hkv=4, d=128, page=64, mix=18),
        # sliding-window decode at head dim 64, small pages
        _case("attend", "attend_window_d64", n=128, ctx=16383, new=1, dtype="bf16", hq=32, hkv=8, d=64, page=16,
              window=1024, mix=19),
        # verification of drafted tokens: a few queries for each request, one KV head per query head
        _case("attend", "attend_drafts", n=32, ctx=2047, new=6, dtype="f16", hq=32, hkv=32, d=128, page=32, mix=20),
        # chunks of long prompts against what is cached of them
        _case("attend", "attend_prompt_chunk", n=2, ctx=14336, new=2048, dtype="bf16", hq=32, hkv=8, d=128, page=64,
              mix=21),
        # cross attention: decoder prompts to encoder states of another length, which are cached once
        _case("attend", "attend_cross", n=16, ctx=1500, new=224, dtype="f16", hq=16, hkv=16, d=64, page=64,
              causal=False, mix=22),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    big = {c["name"]: work(c) for c in listed()}
    while True:
        op = rng.choice(["tables", "write", "attend", "attend"])
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16])
        c = _case(op, n=log(1, 300), ctx=log(1, 100000), new=rng.choice([1, 1, log(2, 16), log(2, 2048)]),
                  dtype=rng.choice(["f16", "bf16"]), hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), hkv=hkv, d=d,
                  page=rng.choice([16, 32, 64, 128]), causal=rng.random() < 0.8, mix=rng.randrange(1, 1 << 20))
        if c["causal"] and rng.random() < 0.3:
            c["window"] = log(16, 8192)
        if not c["causal"]:
            c["ctx"] = min(c["ctx"], 4096)
        ctx, new, kv = _lens(c)
        padded = c["n"] * c["ctx"] * c["hkv"] * c["d"]  # what the padded plain form holds of K
        scores = c["n"] * c["hq"] * c["new"] * (c["ctx"] + c["new"])
        w = work(c)
        if op == "tables":
            ok = c["n"] * c["ctx"] <= 97 * 16384 and sum(new) <= 97 * 1024
        elif op == "write":
            ok = w["bytes"] <= big["write_prompts"]["bytes"] and sum(kv) * hkv * d <= 1 << 28
        else:
            ok = (w["bytes"] <= big["attend_decode"]["bytes"] and w["flops"] <= big["attend_prompt_chunk"]["flops"]
                  and padded <= 1 << 30 and scores <= 1 << 31)
        if ok:
            return c


def _lens(c):
    """Cached tokens before the call, new tokens, and key lengths, by the case alone."""
    r = random.Random(c["mix"])
    n = c["n"]
    ctx = [c["ctx"]] + [r.randint(0, c["ctx"]) for _ in range(n - 1)]
    new = [c["new"]] + [r.randint(1, c["new"]) for _ in range(n - 1)]
    if not c["causal"]:
        ctx = [max(1, x) for x in ctx]
        return ctx, new, ctx
    return ctx, new, [a + b for a, b in zip(ctx, new)]


def _visible_pairs(c):
    """(query, key) pairs of all requests, and keys that some query sees."""
    pairs = keys = 0
    for L, m in zip(*(_lens(c)[i] for i in (2, 1))):
        if not c["causal"]:
            pairs, keys = pairs + m * L, keys + L
            continue
        pos = np.arange(L - m, L, dtype=np.int64)
        lo = np.maximum(0, pos - c["window"] + 1) if c["window"] > 0 else np.zeros_like(pos)
        pairs += int((pos + 1 - lo).sum())
        keys += int(L - lo.min())
    return pairs, keys


def work(c):
    ctx, new, kv = _lens(c)
    T, n, p = sum(new), c["n"], c["page"]
    if c["op"] == "tables":
        fresh = sum((a + b + p - 1) // p - (a + p - 1) // p for a, b in zip(ctx, new))
        # lengths in, ranges and lengths out, slots and positions out, each fresh page's entry in and out
        return {"bytes": 4 * (2 * n + 2 * n + 2 * T + 2 * fresh), "flops": 0}
    if c["op"] == "write":
        # two tensors, 2 bytes in and 1 byte out a value, the slots, a scale for each page touched
        pages = sum((a + b + p - 1) // p - a // p for a, b in zip(ctx, new))
        return {"bytes": 2 * T * c["hkv"] * c["d"] * 3 + 4 * T + 2 * 4 * pages * c["hkv"], "flops": 0}
    pairs, keys = _visible_pairs(c)
    pages = (keys + p - 1) // p
    nbytes = 2 * keys * c["hkv"] * c["d"] + 2 * 4 * pages * c["hkv"] + 4 * pages  # cache, scales, table
    nbytes += T * c["hq"] * (c["d"] * 2 * 2 + 4)  # q, o, lse
    return {"bytes": nbytes, "flops": 4 * c["d"] * c["hq"] * pairs}


def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt * 7919) & 0x7FFFFFFF)


def _cache(shape, seed, salt):
    """Pages of 8-bit values with their scales: normal values whose size differs
    from head to head, as projections of trained weights have it."""
    nb, p, h, d = shape
    g = _gen(seed, salt)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    size = torch.exp2(torch.empty(h, device="cuda").uniform_(-2, 2, generator=g)).to(torch.float16)
    x *= size[None, None, :, None]
    scale = _pow2_scale(x.abs().amax(dim=(1, 3)).float())
    x /= scale.to(torch.float16)[:, None, :, None]
    return x.to(torch.float8_e4m3fn), scale


def _tables(c, seed):
    """Block table of every request's pages (-1 behind them), in shuffled blocks."""
    ctx, new, kv = _lens(c)
    if c["op"] == "tables":  # the new tokens get pages, whatever attends to them
        kv = [x + y for x, y in zip(ctx, new)]
    p = c["page"]
    need = [(max(a, b) + p - 1) // p for a, b in zip(ctx, kv)]
    total = sum(need)
    nb = total + 7
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(nb).astype(np.int32)
    table = np.full((c["n"], max(need)), -1, np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = order[at:at + m]
        at += m
    return table, nb, order


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def prepare(c, seed):
    ctx, new, kv = _lens(c)
    p, T = c["page"], sum(new)
    table, nb, order = _tables(c, seed)
    s = dict(c=c, page=p, T=T, n=c["n"], nb=nb)
    if c["op"] == "tables":
        # the pages of the cached tokens are in the table, the others on the free list
        for r, a in enumerate(ctx):
            table[r, (a + p - 1) // p:] = -1
        used = np.zeros(nb + 1, bool)
        used[table.ravel()] = True
        free = order[~used[order]]
        s.update(ctx=_i32(ctx), new=_i32(new), table=_i32(table), free=_i32(free))
        return s
    if c["op"] == "write":
        slots = []
        for r in range(c["n"]):
            pos = np.arange(ctx[r], ctx[r] + new[r]) if c["causal"] else np.arange(0, min(new[r], kv[r]))
            slots.append(table[r, pos // p] * p + pos % p)
        s["slots"] = _i32(np.concatenate(slots))
        s["T"] = T = s["slots"].numel()
        s["k_cache"], s["k_scale"] = _cache((nb, p, c["hkv"], c["d"]), seed, 1)
        s["v_cache"], s["v_scale"] = _cache((nb, p, c["hkv"], c["d"]), seed, 2)
        for i, x in enumerate(("k", "v")):
            s[x] = torch.randn((1, T, c["hkv"], c["d"]), generator=_gen(seed, 3 + i), device="cuda").to(DT[c["dtype"]])
        return s
    s["k_cache"], s["k_scale"] = _cache((nb, p, c["hkv"], c["d"]), seed, 1)
    s["v_cache"], s["v_scale"] = _cache((nb, p, c["hkv"], c["d"]), seed, 2)
    s["q"] = torch.randn((1, T, c["hq"], c["d"]), generator=_gen(seed, 5), device="cuda").to(DT[c["dtype"]])
    s.update(table=_i32(table), kv=_i32(kv), cu=_i32(np.concatenate([[0], np.cumsum(new)])), new_max=max(new),
             kv_max=max(kv), sm_scale=c["d"] ** -0.5)
    return s


# ------------------------------------------------------------------ the plain forms


def _pow2_scale(amax):
    """The least power of two s (at least 2^-100) with amax <= 448 s; 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_tables(s):
    p, n, T = s["page"], s["n"], s["T"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    cu = torch.zeros(n + 1, dtype=torch.int64, device=table.device)
    torch.cumsum(new, 0, out=cu[1:])
    before, after = (ctx + p - 1) // p, (ctx + new + p - 1) // p
    need = after - before
    first = torch.cumsum(need, 0) - need  # place of the request's first page on the free list
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    take = (first[:, None] + col - before[:, None]).clamp(0, max(0, free.numel() - 1))
    fresh = (col >= before[:, None]) & (col < after[:, None])
    table.copy_(torch.where(fresh, free[take], table))
    t = torch.arange(T, device=table.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    pos = ctx[r] + t - cu[r]
    slot = table[r, pos // p] * p + pos % p
    counts = torch.stack([cu[-1], need.sum(), torch.zeros_like(cu[-1])])
    return [table, cu.int(), (ctx + new).int(), slot.int(), pos.int(), counts.int()]


def _plain_write_one(x, slots, cache, scale):
    nb, p, h, d = cache.shape
    x = x[0].float()
    slots = slots.long()
    page, off = slots // p, slots % p
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    first = torch.full((nb,), p, dtype=torch.int64, device=x.device).index_reduce_(0, page, off, "amin")
    want = _pow2_scale(amax)
    held = (first > 0)[:, None]  # tokens before the first new one stay
    now = torch.where((first < p)[:, None], torch.where(held, torch.maximum(scale, want), want), scale)
    grown = torch.nonzero(((now > scale) & held & (first < p)[:, None]).any(1))[:, 0]
    old = cache.view(torch.uint8)[grown].view(torch.float8_e4m3fn)
    again = (old.float() * (scale[grown] / now[grown])[:, None, :, None]).to(torch.float8_e4m3fn)
    keep = torch.arange(p, device=x.device)[None, :, None, None] < first[grown][:, None, None, None]
    cache.view(torch.uint8)[grown] = torch.where(keep, again.view(torch.uint8), old.view(torch.uint8))
    y = (x / now[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    cache.view(torch.uint8)[page, off] = y.view(torch.uint8)
    scale.copy_(now)


def _plain_write(s):
    _plain_write_one(s["k"], s["slots"], s["k_cache"], s["k_scale"])
    _plain_write_one(s["v"], s["slots"], s["v_cache"], s["v_scale"])
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _gathered(cache, scale, table):
    """[n, KV heads, keys, d] f32 of every request's pages."""
    x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    x *= scale[table][:, :, None, :, None]
    n, m, p, h, d = x.shape
    return x.view(n, m * p, h, d).transpose(1, 2)


def _plain_attend(s):
    c, q = s["c"], s["q"][0]
    T, hq, d = q.shape
    hkv, g, n, m = c["hkv"], hq // c["hkv"], s["n"], s["new_max"]
    p, kv, cu = s["page"], s["kv"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)
    qp = q[rows].float().view(n, m, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * g, d)
    # the pages that a request's queries can see: all of them, or the window's
    pages = (s["kv_max"] + p - 1) // p
    first = torch.zeros_like(kv)
    if c["window"] > 0:
        first = (kv - new - c["window"] + 1).clamp(min=0) // p
        pages = min(pages, (c["window"] + m - 2) // p + 2)
    col = first[:, None] + torch.arange(pages, device=q.device)
    table = s["table"].long().gather(1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    j = (first * p)[:, None] + torch.arange(pages * p, device=q.device)
    k = _gathered(s["k_cache"], s["k_scale"], table)
    L = k.shape[2]
    see = (j < kv[:, None])[:, None, :]
    if c["causal"]:
        pos = ((kv - new)[:, None] + i[None, :])[:, :, None]
        see = see & (j[:, None, :] <= pos)
        if c["window"] > 0:
            see = see & (j[:, None, :] > pos - c["window"])
    else:
        see = see.expand(n, m, L)
    x = torch.matmul(qp, k.transpose(2, 3)).mul_(s["sm_scale"]).view(n, hkv, m, g, L)
    del k
    x.masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scale"], table)
    o = torch.matmul(x.view(n, hkv, m * g, L), v).view(n, hkv, m, g, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (total.log() + top)[..., 0]
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    o = o[r, :, t - cu[r]].reshape(1, T, hq, d).to(q.dtype)
    lse = lse[r, :, t - cu[r]].reshape(1, T, hq).transpose(1, 2).contiguous()
    return [o, lse]


def run(s):
    c = s["c"]
    if own:
        import attention_backward_gb300 as ab

        if c["op"] == "tables":
            plan = ab.kv_block_tables(s["ctx"], s["new"], s["table"], s["free"], s["page"], s["nb"], s["T"])
            return [s["table"], plan.cu_seqlens, plan.kv_lens, plan.slot_map, plan.positions, plan.counts]
        if c["op"] == "write":
            ab.kv_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
            return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
        return list(ab.forward_kv_cache(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                        s["cu"], s["kv"], s["sm_scale"], causal=c["causal"], window=c["window"]))
    return {"tables": _plain_tables, "write": _plain_write, "attend": _plain_attend}[c["op"]](s)


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _e4m3(x):
    """x (f64) at the nearest e4m3 value, ties to the even one: steps of 2^-9 below 2^-6, of an eighth of the binade above."""
    a = x.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _exact_tables(s):
    p = s["page"]
    ctx, new, table, free = (s[x].cpu().tolist() for x in ("ctx", "new", "table", "free"))
    cu, slots, positions, taken = [0], [], [], 0
    for a, b, row in zip(ctx, new, table):
        for j in range(-(-a // p), -(-(a + b) // p)):
            row[j] = free[taken]
            taken += 1
        for pos in range(a, a + b):
            slots.append(row[pos // p] * p + pos % p)
            positions.append(pos)
        cu.append(cu[-1] + b)
    got = [table, cu, [a + b for a, b in zip(ctx, new)], slots, positions, [cu[-1], taken, 0]]
    return [np.asarray(x, dtype=np.int32) for x in got]


def _exact_write_one(x, slots, cache, scale, p):
    values, scales = cache.double(), scale.double()
    x, slots = x[0].double(), slots.cpu().numpy()
    heads = ((slots[1:] != slots[:-1] + 1) | (slots[1:] % p == 0)).nonzero()[0] + 1
    edges = [0, *heads.tolist(), len(slots)]
    for a, b in zip(edges[:-1], edges[1:]):
        page, off = divmod(int(slots[a]), p)
        e = torch.ceil(torch.log2(x[a:b].abs().amax(dim=(0, 2)) / E4M3_MAX)).clamp(min=MIN_EXP)
        now = torch.exp2(e)
        if off:
            now = torch.maximum(now, scales[page])
            values[page, :off] = _e4m3(values[page, :off] * (scales[page] / now)[None, :, None])
        values[page, off:off + b - a] = _e4m3(x[a:b] / now[None, :, None])
        scales[page] = now
    return values, scales


def _exact_attend(s):
    c, p, q = s["c"], s["page"], s["q"][0]
    T, hq, d = q.shape
    g = hq // c["hkv"]
    o = torch.zeros(1, T, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((1, hq, T), -math.inf, dtype=torch.float64, device=q.device)
    cu, kv, table = s["cu"].tolist(), s["kv"].tolist(), s["table"].tolist()
    for r, L in enumerate(kv):
        if L == 0 or cu[r + 1] == cu[r]:
            continue
        a, m = cu[r], cu[r + 1] - cu[r]
        blocks = torch.tensor(table[r][:(L + p - 1) // p], device=q.device)
        see = torch.ones(m, L, dtype=torch.bool, device=q.device)
        if c["causal"]:
            far = (torch.arange(m, device=q.device)[:, None] + (L - m)) - torch.arange(L, device=q.device)[None, :]
            see = (far >= 0) & ((far < c["window"]) if c["window"] > 0 else (far >= 0))
        for h in range(c["hkv"]):
            ks, vs = (s[x + "_cache"].view(torch.uint8)[blocks, :, h].view(torch.float8_e4m3fn).double() *
                      s[x + "_scale"][blocks, h].double()[:, None, None] for x in ("k", "v"))
            ks, vs = ks.reshape(-1, d)[:L], vs.reshape(-1, d)[:L]
            for f in range(h * g, (h + 1) * g):
                w = q[a:a + m, f].double() @ ks.T * s["sm_scale"]
                w = w.masked_fill(~see, -math.inf)
                z = torch.logsumexp(w, -1)
                lse[0, f, a:a + m] = z
                o[0, a:a + m, f] = torch.exp(w - z[:, None]) @ vs
    return [o, lse]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "tables":
        return _exact_tables(s)
    if c["op"] == "write":
        kc, ks = _exact_write_one(s["k"], s["slots"], s["k_cache"], s["k_scale"], s["page"])
        vc, vs = _exact_write_one(s["v"], s["slots"], s["v_cache"], s["v_scale"], s["page"])
        return [kc, vc, ks, vs]
    return _exact_attend(s)
