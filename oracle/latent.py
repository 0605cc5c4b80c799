"""Float64 definitions of rotary positions and latent attention, on the CPU.

The attention functions return, beside O and the LSE, what tolerances are made of:
per element of O the sum of p |v| and the error that errors e_j of the weights'
exponents make, sum p e |v| + |o| sum p e; per row sum p e; and per element the sum of
|v| over the row's keys.  e_j = D 2^-23 sum |q||k_j| scale + 2^-21: f32 sums of D
products, the rounding of the scaled score and of its power.
"""
import numpy as np

LAT, ROT = 512, 64


def turn(x, start, freqs, pos, scale=1.0, interleaved=False, inverse=False):
    """x [..., D] with columns [start, start + 2 len(freqs)) turned to ``pos``
    (broadcast against x's leading dimensions), and |x1| + |x2| of each element's pair
    (0 outside those columns)."""
    R = 2 * len(freqs)
    t = np.asarray(pos, dtype=np.float64)[..., None] * np.asarray(freqs) * (-1 if inverse else 1)
    i = np.arange(R // 2)
    a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + i + R // 2)
    y, size = x.astype(np.float64).copy(), np.zeros(x.shape)
    x1, x2 = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
    y[..., a] = scale * (x1 * np.cos(t) - x2 * np.sin(t))
    y[..., b] = scale * (x1 * np.sin(t) + x2 * np.cos(t))
    size[..., a] = size[..., b] = np.abs(x1) + np.abs(x2)
    return y, size


def cache_rows(kv, weight=None, eps=0.0, freqs=None, pos=None, scale=1.0, interleaved=False):
    """Rows (c' | k') of kv [T, 576], and the size of each element's pair (of c': of itself)."""
    y, size = kv.astype(np.float64).copy(), np.abs(kv.astype(np.float64))
    if freqs is not None:
        y, pair = turn(kv, LAT, freqs, pos, scale, interleaved)
        size[:, LAT:] = pair[:, LAT:] * abs(scale)
    if weight is not None:
        c = kv[:, :LAT].astype(np.float64)
        y[:, :LAT] = c / np.sqrt((c * c).mean(1, keepdims=True) + eps) * weight
        size[:, :LAT] = np.abs(y[:, :LAT])
    return y, size


class Result:
    """O, LSE and the tolerances' parts, of rows laid out as ``shape`` (+ value columns)."""

    def __init__(self, shape, dv, fill=np.nan):
        self.o = np.full((*shape, dv), fill)
        self.lse = np.full(shape, fill)
        self.mag, self.oe, self.low = (np.zeros((*shape, dv)) for _ in range(3))
        self.le, self.seen = np.zeros(shape), np.zeros(shape)

    def put(self, at, q, k, v, scale, see=None):
        """Rows ``at`` are softmax(scale q k^T) v over the keys that ``see`` marks."""
        q, k, v = (x.astype(np.float64) for x in (q, k, v))
        see = np.ones((len(q), len(k)), bool) if see is None else see
        x = np.where(see, scale * (q @ k.T), -np.inf)
        top = x.max(1, initial=-np.inf, keepdims=True)
        top = np.where(np.isneginf(top), 0, top)
        p = np.exp(x - top)
        total = p.sum(1, keepdims=True)
        with np.errstate(divide="ignore"):
            self.lse[at] = (top + np.log(total))[:, 0]
        p /= np.where(total > 0, total, 1)
        e = q.shape[1] * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(k).T) + 2.0 ** -21
        self.o[at], self.mag[at] = p @ v, p @ np.abs(v)
        self.le[at] = (p * e).sum(1)
        self.oe[at] = (p * e) @ np.abs(v) + np.abs(self.o[at]) * (p * e).sum(1, keepdims=True)
        self.low[at] = see.astype(np.float64) @ np.abs(v)
        self.seen[at] = see.sum(1)


def cache_forward(q, cache, table, cu, kv_lens, scale, causal=True):
    """q [T, H, 576] over cache [num_blocks, page, 576]; rows of no request stay NaN."""
    T, H, _ = q.shape
    nb, P, _ = cache.shape
    r = Result((T, H), LAT)
    for n, length in enumerate(kv_lens):
        a, e = max(0, min(T, int(cu[n]))), max(0, min(T, int(cu[n + 1])))
        m, length = e - a, max(0, int(length))
        if m <= 0:
            continue
        pos = np.arange(min(length, table.shape[1] * P))
        blk = table[n, pos // P]
        see = np.broadcast_to((blk >= 0) & (blk < nb), (m, len(pos))).copy()
        if causal:
            see &= pos[None, :] <= np.arange(m)[:, None] + length - m
        some = see.any(0)
        k = np.where(some[:, None], cache[np.where(some, blk, 0), pos % P], 0)
        for h in range(H):
            r.put((slice(a, e), h), q[a:e, h], k, k[:, :LAT], scale, see)
    return r


def list_forward(q, kv, idx, scale):
    """q [B, S, H, 576], kv [B, SKV, HKV, 576], idx [B, S, HKV, topk]."""
    B, S, H, _ = q.shape
    SKV, HKV = kv.shape[1:3]
    G = H // HKV
    r = Result((B, S, H), LAT)
    for b in range(B):
        for t in range(S):
            for g in range(HKV):
                k = kv[b, idx[b, t, g][(idx[b, t, g] >= 0) & (idx[b, t, g] < SKV)], g]
                r.put((b, t, slice(g * G, (g + 1) * G)), q[b, t, g * G:(g + 1) * G], k, k[:, :LAT], scale)
    return r


def expanded_forward(q, kn, kr, v, scale, causal=True, cu=None):
    """q [B, S, H, 192], kn, v [B, Sk, H, 128], kr [B, Sk, 64]; rows of no sequence stay NaN."""
    B, S, H, _ = q.shape
    Sk = kn.shape[1]
    r = Result((B, S, H), v.shape[3])
    seqs = [(0, S, 0, Sk)] if cu is None else [(a, e, a, e) for a, e in zip(cu[:-1], cu[1:])]
    for b in range(B):
        for a, e, ka, ke in seqs:
            if e <= a:
                continue
            off = (ke - ka) - (e - a)
            see = np.ones((e - a, ke - ka), bool)
            if causal:
                see = np.arange(ke - ka)[None, :] <= np.arange(e - a)[:, None] + off
            for h in range(H):
                k = np.concatenate([kn[b, ka:ke, h], kr[b, ka:ke]], 1)
                r.put((b, slice(a, e), h), q[b, a:e, h], k, v[b, ka:ke, h], scale, see)
    return r
