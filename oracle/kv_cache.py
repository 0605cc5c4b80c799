"""The paged 8-bit cache operators in float64 (test infrastructure only).

Plain restatements of the definitions in ``include/attn_kv_cache.h``, one
request, run, page or head at a time.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _e4m3_values() -> np.ndarray:
    """The value of each byte: (-1)^s 2^(e - 7) (1 + f/8), subnormal steps of 2^-9, 0x7f and 0xff NaN."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(1.0 + f / 8.0, e - 7), f * 2.0 ** -9)
    v[(b & 127) == 127] = np.nan
    return np.where(b & 128, -v, v)


E4M3 = _e4m3_values()


def to_e4m3(x) -> np.ndarray:
    """Bytes of the nearest e4m3 values (ties to the even fraction, +-448 beyond, NaN 0x7f)."""
    x = np.asarray(x, dtype=np.float64)
    grid = E4M3[:127]  # ascending from 0 to 448
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=E4M3_MAX, neginf=-E4M3_MAX)), E4M3_MAX)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    out = pick | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, out).astype(np.uint8)


def scale_for(amax: float) -> float:
    """The least power of two s >= 2^-100 with amax <= 448 s."""
    s = 2.0 ** -100
    while amax > E4M3_MAX * s:
        s *= 2.0
    return s


def block_tables(ctx, new, table, free, page, num_blocks, max_tokens, start=0):
    """(table, cu_seqlens, kv_lens, slot_map, positions, counts)."""
    table = np.array(table, dtype=np.int64)
    ctx, new = [max(0, int(x)) for x in ctx], [max(0, int(x)) for x in new]
    width = table.shape[1]
    taken = lacking = 0
    given = [b if 0 <= b < num_blocks else -1 for b in list(free)[max(0, start):]]
    cu, slots, positions = [0], [], []
    for n, (a, b) in enumerate(zip(ctx, new)):
        for j in range(-(-a // page), -(-(a + b) // page)):
            if j >= width:
                lacking += 1
            elif taken < len(given):
                table[n, j] = given[taken]
                taken += 1
            else:
                table[n, j] = -1
                lacking += 1
        for pos in range(a, a + b):
            blk = table[n, pos // page] if pos // page < width else -1
            slots.append(blk * page + pos % page if 0 <= blk < num_blocks else -1)
            positions.append(pos)
        cu.append(cu[-1] + b)
    counts = [cu[-1], taken, lacking + max(0, cu[-1] - max_tokens)]
    pad = max(0, max_tokens - len(slots))
    slots, positions = slots[:max_tokens] + [-1] * pad, positions[:max_tokens] + [0] * pad
    return (table, np.minimum(cu, max_tokens), np.array(ctx) + np.array(new), np.array(slots, dtype=np.int64),
            np.array(positions, dtype=np.int64), np.array(counts))


def write(x, slots, cache, scale):
    """New (cache bytes [blocks, P, H, D], scale [blocks, H]) with tokens x [T,H,D] at ``slots``."""
    cache, scale = cache.copy(), scale.astype(np.float64).copy()
    nb, P, H, D = cache.shape
    tokens = [t for t, s in enumerate(slots) if 0 <= s < nb * P]
    runs: list = []
    for t in tokens:
        if runs:
            u = runs[-1][-1]
            if t - u <= 32 and slots[u] // P == slots[t] // P and slots[u] < slots[t]:
                runs[-1].append(t)
                continue
        runs.append([t])
    for r in runs:
        s = int(slots[r[0]])
        blk, off = divmod(s, P)
        for h in range(H):
            run = x[r, h].astype(np.float64)
            fin = np.abs(run[np.isfinite(run)])
            want = scale_for(fin.max() if fin.size else 0.0)
            old = scale[blk, h]
            now = want
            if off and old >= want:
                now = old
            elif off and want > old:
                cache[blk, :off, h] = to_e4m3(E4M3[cache[blk, :off, h]] * (old / now))
            scale[blk, h] = now
            with np.errstate(invalid="ignore"):
                cache[blk, [int(slots[t]) % P for t in r], h] = to_e4m3(run / now)
    return cache, scale


def forward(q, k_cache, v_cache, k_scale, v_scale, table, cu, kv_lens, scale, causal, window):
    """O [T,HQ,D], LSE [HQ,T], and what their tolerances are made of: the sum of
    p |v| per element of O, the largest |q| . |k| of each row times ``scale``,
    the keys each row sees and the largest |v| among them.  Rows of no request
    stay NaN."""
    T, HQ, D = q.shape
    nb, P, HKV, _ = k_cache.shape
    G = HQ // HKV
    o, mag = np.full((T, HQ, D), np.nan), np.zeros((T, HQ, D))
    lse, dots = np.full((HQ, T), np.nan), np.zeros((HQ, T))
    seen, vmax = np.zeros((HQ, T)), np.zeros((HQ, T))
    for n in range(len(kv_lens)):
        a, e = max(0, min(T, int(cu[n]))), max(0, min(T, int(cu[n + 1])))
        m, length = e - a, max(0, int(kv_lens[n]))
        if m <= 0:
            continue
        L = min(length, table.shape[1] * P)  # positions that the table holds
        pos = np.arange(L)
        page = pos // P
        blk = table[n, page]
        held = (blk >= 0) & (blk < nb)
        i = np.arange(m)[:, None] + length - m
        see = np.broadcast_to(held, (m, L)).copy()
        if causal or window > 0:
            see &= pos[None, :] <= i
        if window > 0:
            see &= pos[None, :] > i - window
        any_row = see.any(0)
        b = np.where(any_row, blk, 0)
        for h in range(HKV):
            with np.errstate(invalid="ignore"):
                K = np.where(any_row[:, None], E4M3[k_cache[b, pos % P, h]] * k_scale[b, h].astype(np.float64)[:, None], 0)
                V = np.where(any_row[:, None], E4M3[v_cache[b, pos % P, h]] * v_scale[b, h].astype(np.float64)[:, None], 0)
            for f in range(h * G, (h + 1) * G):
                Q = q[a:e, f].astype(np.float64)
                s = np.where(see, (Q @ K.T) * scale, -np.inf)
                mx = s.max(1, initial=-np.inf, keepdims=True)
                mx = np.where(np.isfinite(mx), mx, 0)
                p = np.exp(s - mx)
                tot = p.sum(1, keepdims=True)
                with np.errstate(divide="ignore"):
                    lse[f, a:e] = (mx + np.log(tot))[:, 0]
                p = p / np.where(tot > 0, tot, 1)
                o[a:e, f], mag[a:e, f] = p @ V, p @ np.abs(V)
                if L:
                    dots[f, a:e] = np.where(see, (np.abs(Q) @ np.abs(K).T) * scale, 0).max(1)
                    seen[f, a:e] = see.sum(1)
                    vmax[f, a:e] = np.where(see, np.abs(V).max(1), 0).max(1)
    return o, lse, mag, dots, seen, vmax
