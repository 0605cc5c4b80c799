"""GPU parity of the paged 8-bit cache operators with their float64 oracle:
block tables and slots exactly, cache bytes and scales exactly, attention within
a bound made from the arithmetic.

The bound of O, element by element, with p the normalised weights:
  eps/2 |o|                    the rounding of the output
  (2^-11 + e) sum p |v|        fp16 rounding of P, and the error e of the
                               weights' exponents
  2^-24 n vmax                 P below fp16's normal range (2^-25 a key, and
                               448 times a page's scale is under 2 vmax)
with e = 2 (D 2^-23 sum |q||k| scale + 2^-21): f32 sums of D products and the
rounding of the scaled score, for the numerator and the denominator.  The LSE
has e + 2^-23 |lse| + 2^-20 (f32 sum and logarithm).
"""
import numpy as np
import pytest

from oracle import kv_cache as oracle

pytestmark = pytest.mark.gpu


def cuda(x, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(x):
    return cuda(np.asarray(x, dtype=np.int32))


def dt_of(name):
    import torch

    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def rounded(rng, shape, name, size=1.0):
    """Normal values of a 16-bit type, as float64."""
    import torch

    return torch.from_numpy(rng.standard_normal(shape) * size).to(dt_of(name)).double().numpy()


def fp8(b, heads_first=False):
    import torch

    t = torch.from_numpy(b.copy()).cuda()
    if heads_first:
        t = t.transpose(1, 2).contiguous().transpose(1, 2)
    return t.view(torch.float8_e4m3fn)


def bytes_of(t):
    import torch

    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ block tables


def tables_problem(n, page, hi_ctx, hi_new, seed, spare=3):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, hi_ctx + 1, n), rng.integers(0, hi_new + 1, n)
    ctx[rng.random(n) < 0.3] //= page
    ctx[rng.random(n) < 0.3] = ctx[rng.random(n) < 0.3].size % (hi_ctx + 1)
    before, after = -(-ctx // page), -(-(ctx + new) // page)
    nb = int(after.sum()) + spare
    order = rng.permutation(nb)
    table = np.full((n, int(after.max()) + 2), -1)
    at = 0
    for r in range(n):
        table[r, :before[r]] = order[at:at + before[r]]
        at += before[r]
    return ctx, new, table, order[at:], nb


def run_tables(ctx, new, table, free, page, nb, T, start=None, poison=True):
    import torch

    import attention_backward_gb300 as ab

    n = len(ctx)
    out = None
    if poison:
        out = ab.KvPlan(*(torch.full((k,), -77, dtype=torch.int32, device="cuda") for k in (n + 1, n, T, T, 3)))
    t = i32(table)
    plan = ab.kv_block_tables(i32(ctx), i32(new), t, i32(free), page, nb, T,
                              free_start=None if start is None else i32([start]), out=out)
    return [t.cpu().numpy()] + [x.cpu().numpy() for x in plan]


def same_plan(got, ref):
    for name, g, r in zip(("table", "cu_seqlens", "kv_lens", "slot_map", "positions", "counts"), got, ref):
        assert np.array_equal(g, r), (name, g, r)


@pytest.mark.parametrize("n,page,hi_ctx,hi_new,pad", [
    (1, 16, 0, 1, 0), (1, 64, 200, 300, 5), (7, 16, 100, 1, 0), (33, 32, 70, 40, 11), (256, 16, 500, 1, 0),
    (511, 128, 300, 3, 1), (513, 16, 50, 2, 0), (1500, 64, 130, 70, 100), (3, 128, 5000, 4000, 0)])
def test_block_tables(n, page, hi_ctx, hi_new, pad):
    ctx, new, table, free, nb = tables_problem(n, page, hi_ctx, hi_new, 100 + n)
    T = int(new.sum()) + pad
    ref = oracle.block_tables(ctx, new, table, free, page, nb, T)
    same_plan(run_tables(ctx, new, table, free, page, nb, T), ref)
    same_plan(run_tables(ctx, new, table, free, page, nb, T, poison=False), ref)


def test_block_tables_free_start_and_negative_lengths():
    ctx, new, table, free, nb = tables_problem(40, 32, 100, 90, 5)
    ctx[3], new[4], new[7] = -5, -1, 0
    table[3] = -1
    skipped = np.concatenate([[nb + 50] * 9, free])  # entries before free_start are not looked at
    T = int(np.maximum(new, 0).sum())
    ref = oracle.block_tables(ctx, new, table, skipped, 32, nb, T, start=9)
    assert ref[5][2] == 0
    same_plan(run_tables(ctx, new, table, skipped, 32, nb, T, start=9), ref)


@pytest.mark.parametrize("what", ["pages", "start", "width", "tokens", "entries", "none"])
def test_block_tables_that_do_not_fit(what):
    ctx, new, table, free, nb = tables_problem(50, 16, 100, 60, 6)
    T, start = int(new.sum()), None
    if what == "pages":
        free = free[:len(free) // 2]
    elif what == "none":
        free = free[:0]
    elif what == "start":
        start = len(free) + 4
    elif what == "width":
        table = table[:, :4]
    elif what == "tokens":
        T = T // 2
    else:
        free = free.copy()
        free[::3], free[1::3] = -4, nb
    ref = oracle.block_tables(ctx, new, table, free, 16, nb, T, start=start or 0)
    if what != "entries":
        assert ref[5][2] > 0
    same_plan(run_tables(ctx, new, table, free, 16, nb, T, start=start), ref)


def test_block_tables_leave_other_entries_alone():
    ctx, new, table, free, nb = tables_problem(64, 16, 100, 60, 8)
    table[table < 0] = 12345
    ref = oracle.block_tables(ctx, new, table, free, 16, nb, int(new.sum()))
    assert (ref[0] == 12345).any()
    same_plan(run_tables(ctx, new, table, free, 16, nb, int(new.sum())), ref)


# ------------------------------------------------------------------ cache writes


def write_problem(name, T, HKV, D, page, hi_new, seed, size=1.0):
    """Requests of 1 to hi_new new tokens that start anywhere in a page; the
    cache holds finite values, as earlier steps left them."""
    rng = np.random.default_rng(seed)
    slots, blk = [], 0
    while len(slots) < T:
        m = int(min(rng.integers(1, hi_new + 1), T - len(slots)))
        off = int(rng.integers(0, page)) if rng.random() < 0.7 else 0
        slots += [blk * page + off + i for i in range(m)]
        blk = slots[-1] // page + 1
    nb = blk + 2
    perm = rng.permutation(nb)
    slots = np.array([perm[s // page] * page + s % page for s in slots])
    x = [rounded(rng, (T, HKV, D), name, size * 2.0 ** rng.integers(-3, 4)) for _ in range(2)]
    cache = [oracle.to_e4m3(rng.standard_normal((nb, page, HKV, D)) * 100) for _ in range(2)]
    scale = [np.exp2(rng.integers(-12, -2, (nb, HKV))) for _ in range(2)]
    return x, slots, cache, scale


def run_write(x, slots, cache, scale, name, heads_first=False, fused=False):
    import torch

    import attention_backward_gb300 as ab

    tx = [cuda(a, dt_of(name))[None] for a in x]
    if fused:  # keys and values as slices of one projection's rows
        both = torch.full((1, x[0].shape[0], 2 * x[0].shape[1] + 1, x[0].shape[2]), float("nan"), dtype=dt_of(name),
                          device="cuda")
        H = x[0].shape[1]
        both[:, :, :H], both[:, :, H + 1:] = tx[0], tx[1]
        tx = [both[:, :, :H], both[:, :, H + 1:]]
    tc = [fp8(c, heads_first) for c in cache]
    ts = [cuda(s.astype(np.float32)) for s in scale]
    ab.kv_cache_write(tx[0], tx[1], i32(slots), tc[0], tc[1], ts[0], ts[1])
    return [bytes_of(t) for t in tc], [t.double().cpu().numpy() for t in ts]


def check_write(x, slots, cache, scale, name, **kw):
    import torch

    x = [torch.from_numpy(a).to(dt_of(name)).double().numpy() for a in x]  # the values that the kernel gets
    gc, gs = run_write(x, slots, cache, scale, name, **kw)
    for i in range(2):
        rc, rs = oracle.write(x[i], slots, cache[i], scale[i])
        assert np.array_equal(gs[i], rs.astype(np.float32).astype(np.float64)), ("scale", i)
        same = (gc[i] == rc) | (np.isnan(oracle.E4M3[gc[i]]) & np.isnan(oracle.E4M3[rc]))
        assert same.all(), (i, np.argwhere(~same)[:5])


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("T,HKV,D,page,hi_new", [
    (1, 1, 64, 16, 1), (1, 8, 128, 128, 1), (5, 3, 128, 16, 1), (64, 8, 128, 64, 1), (67, 2, 64, 32, 5),
    (300, 5, 128, 128, 290), (1023, 1, 64, 16, 200), (4097, 2, 64, 64, 900), (4200, 4, 128, 128, 50),
    (4099, 7, 64, 16, 1)])
def test_cache_write(name, T, HKV, D, page, hi_new):
    check_write(*write_problem(name, T, HKV, D, page, hi_new, T + D), name)


@pytest.mark.parametrize("kw", [dict(heads_first=True), dict(fused=True), dict(heads_first=True, fused=True)])
def test_cache_write_of_other_layouts(kw):
    check_write(*write_problem("bf16", 150, 6, 128, 32, 40, 3), "bf16", **kw)


def test_cache_write_skips_slots_outside_the_cache():
    x, slots, cache, scale = write_problem("f16", 90, 2, 64, 16, 7, 4)
    total = cache[0].shape[0] * 16
    slots[5::11], slots[7::13] = -1, total
    slots[-1] = total + 3
    check_write(x, slots, cache, scale, "f16")


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_cache_write_of_special_values(name):
    """Zeros, the type's largest and smallest values, infinities, NaN, ties."""
    import torch

    x, slots, cache, scale = write_problem(name, 48, 2, 64, 16, 9, 5)
    info = torch.finfo(dt_of(name))
    for a in x:
        a[0:4] = 0.0
        a[4, 0, :8] = [np.inf, -np.inf, np.nan, 1, -1, 0.5, 2, 3]
        a[7, 1] = np.inf
        a[9, 1] = np.nan
        a[12, 0, 0] = info.max if name == "f16" else 2.0 ** 110
        a[15] = float(info.smallest_normal) / 8  # a subnormal value
        a[20] = (np.arange(64) % 33)[None] / 16 + 17  # ties between e4m3 steps
        a[24, 1, 0] = 448.0
    check_write(x, slots, cache, scale, name)


def test_cache_write_keeps_a_larger_scale_of_any_value():
    x, slots, cache, scale = write_problem("bf16", 60, 3, 128, 32, 4, 6)
    scale = [s * 3.0 for s in scale]  # not powers of two: kept, and rounded against exactly
    check_write([a * 0.25 for a in x], slots, cache, scale, "bf16")


@pytest.mark.parametrize("page", [16, 64])
def test_cache_write_token_by_token(page):
    """A page filled by single-token calls ends with the scale of one call over
    all its tokens, and with the same values down to the smallest e4m3 step."""
    import attention_backward_gb300 as ab

    rng = np.random.default_rng(9)
    x = rounded(rng, (page, 2, 64), "bf16") * np.exp2(rng.integers(-2, 3, (page, 1, 1)))
    zero = np.zeros((3, page, 2, 64), dtype=np.uint8)
    slots = 2 * page + np.arange(page)
    whole, ws = oracle.write(x, slots, zero, np.zeros((3, 2)))
    tc, ts = [fp8(zero) for _ in range(2)], [cuda(np.zeros((3, 2), np.float32)) for _ in range(2)]
    tx, sl = cuda(x, dt_of("bf16"))[None], i32(slots)
    for t in range(page):
        ab.kv_cache_write(tx[:, t:t + 1], tx[:, t:t + 1], sl[t:t + 1], *tc, *ts)
    for c, s in zip(tc, ts):
        assert np.array_equal(s.double().cpu().numpy(), ws)
        off = np.abs(oracle.E4M3[bytes_of(c)] - oracle.E4M3[whole])
        assert (off <= 2.0 ** -9).all()
        assert (off[np.abs(oracle.E4M3[whole]) >= 2.0 ** -5] == 0).all()


# ------------------------------------------------------------------ attention


def attend_problem(name, lens, HQ, HKV, D, page, seed, spare_rows=0, size=1.0):
    """``lens``: (queries, keys) of each request.  Bytes and scales that no
    request holds are NaN, the table's other entries point nowhere."""
    rng = np.random.default_rng(seed)
    need = [-(-L // page) for _, L in lens]
    nb = sum(need) + 2
    perm = rng.permutation(nb)
    table = np.full((len(lens), max(max(need), 1) + 1), 1 << 30)
    kc, vc = (np.full((nb, page, HKV, D), 0x7F, dtype=np.uint8) for _ in range(2))
    ks, vs = (np.full((nb, HKV), np.nan) for _ in range(2))
    at = 0
    for r, (_, L) in enumerate(lens):
        for j in range(need[r]):
            b = table[r, j] = perm[at]
            at += 1
            m = min(page, L - j * page)
            for c, s in ((kc, ks), (vc, vs)):
                s[b] = np.exp2(rng.integers(-8, -4, HKV))
                c[b, :m] = oracle.to_e4m3(rng.standard_normal((m, HKV, D)) / s[b][None, :, None] * size)
    cu = np.concatenate([[0], np.cumsum([m for m, _ in lens])])
    q = rounded(rng, (int(cu[-1]) + spare_rows, HQ, D), name)
    return q, kc, vc, ks, vs, table, cu, np.array([L for _, L in lens])


def run_attend(prob, name, causal=True, window=-1, scale=None, heads_first=False, workspace=None, stream=None):
    import torch

    import attention_backward_gb300 as ab

    q, kc, vc, ks, vs, table, cu, kv = prob
    tq = cuda(q, dt_of(name))[None]
    o = torch.full_like(tq, float("nan"))
    lse = torch.full((1, q.shape[1], q.shape[0]), float("nan"), device="cuda")
    if workspace is None:
        workspace = torch.full((ab.kv_cache_workspace_size(q.shape[0], q.shape[1], kc.shape[2], q.shape[2]),), 0xFF,
                               dtype=torch.uint8, device="cuda")
    ab.forward_kv_cache(tq, fp8(kc, heads_first), fp8(vc, heads_first), cuda(ks.astype(np.float32)),
                        cuda(vs.astype(np.float32)), i32(table), i32(cu), i32(kv), scale, causal, window, workspace,
                        (o, lse), stream)
    ab.check_error(workspace, stream)
    return o[0].double().cpu().numpy(), lse[0].double().cpu().numpy()


def check_attend(prob, name, causal=True, window=-1, scale=None, v_rounded=False, **kw):
    """v_rounded: many rows and V scales that are no powers of two; their values
    are rounded to fp16 at the largest scale, 2^-11 relative."""
    q, kc, vc, ks, vs, table, cu, kv = prob
    D = q.shape[2]
    got, glse = run_attend(prob, name, causal, window, scale, **kw)
    o, lse, mag, dots, seen, vmax = oracle.forward(q, kc, vc, ks, vs, table, cu, kv, scale or D ** -0.5, causal,
                                                   window)
    live = ~np.isnan(lse)
    assert np.isnan(glse[~live]).all() and np.isnan(got[~live.T]).all()  # rows of no request stay as they were
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(glse), none) and (got[none.T] == 0).all()
    e = 2 * (D * 2.0 ** -23 * dots + 2.0 ** -21)
    some = live & ~none
    tl = (e + 2.0 ** -23 * np.abs(lse) + 2.0 ** -20)[some]
    el = np.abs(glse[some] - lse[some])
    assert (el <= tl).all(), (el / tl).max()
    half = 2.0 ** -11 if name == "f16" else 2.0 ** -8
    tiny = 2.0 ** -25 if name == "f16" else 0.0  # half of fp16's smallest step
    tol = half * np.abs(o) + (2.0 ** -11 * (1 + v_rounded) + e.T[..., None]) * mag * (1 + half) + (2.0 ** -24 * seen * vmax).T[..., None] + tiny
    err = np.abs(got - o)[live.T]
    assert (err <= tol[live.T]).all(), (err / tol[live.T]).max()


DECODE = [
    # lens, HQ, HKV, D, page
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 1)], 8, 8, 128, 128),
    ([(1, 17), (1, 16), (1, 15), (1, 64), (1, 65), (1, 63)], 8, 2, 128, 16),
    ([(1, 333)], 32, 8, 128, 16),
    ([(1, 5000)], 16, 1, 128, 64),
    ([(1, 5000), (1, 1)], 6, 2, 64, 32),
    ([(1, L) for L in (1, 700, 3, 129, 128, 2000, 64, 31)], 12, 4, 64, 128),
    ([(1, 100 + 7 * i) for i in range(150)], 14, 2, 64, 16),  # more requests than threads of a CTA
    ([(1, 900)], 80, 2, 64, 64),  # groups of 40 heads: three row tiles
    ([(2, 300), (1, 2), (5, 5), (3, 1000), (7, 90)], 8, 8, 128, 32),
    ([(3, 700), (6, 129), (1, 64)], 28, 4, 64, 64),
]


@pytest.mark.parametrize("D,page", [(64, 16), (64, 32), (128, 16), (128, 64)])
def test_attend_with_more_heads_than_workers(D, page):
    """2100 KV heads: more than the warps of a launch, so each serves several."""
    check_attend(attend_problem("f16", [(1, 70), (0, 3), (2, 33)], 2100, 2100, D, page, 30), "f16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attend_every_page_size(D, page):
    """Lengths around tiles, blocks and pages, for few rows and for many."""
    few = [(1, L) for L in (15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 255, 257)]
    check_attend(attend_problem("bf16", few, 3, 1, D, page, 31), "bf16")
    check_attend(attend_problem("bf16", few, 3, 1, D, page, 31), "bf16", window=40)
    many = [(70, L) for L in (70, 127, 128, 129, 200, 257)]
    check_attend(attend_problem("bf16", many, 3, 1, D, page, 32), "bf16")
    check_attend(attend_problem("bf16", many, 3, 1, D, page, 32), "bf16", window=40)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_attend(case, name):
    lens, HQ, HKV, D, page = DECODE[case]
    check_attend(attend_problem(name, lens, HQ, HKV, D, page, 40 + case), name)


@pytest.mark.parametrize("causal,window", [(False, -1), (True, 1), (True, 2), (True, 70), (True, 256), (False, 33),
                                           (True, 100000)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_masks(causal, window, D):
    lens = [(1, 1000), (4, 4), (9, 300), (1, 1), (2, 71), (40, 130), (1, 513)]
    check_attend(attend_problem("bf16", lens, 6, 2, D, 16, 7, spare_rows=3), "bf16", causal, window)


PROMPTS = [
    ([(300, 300)], 8, 2, 128, 16),
    ([(257, 900)], 4, 4, 64, 64),
    ([(65, 65)], 1, 1, 128, 128),
    ([(128, 128), (1, 700), (65, 66), (500, 2000), (3, 3), (0, 9)], 6, 2, 128, 32),
    ([(1000, 1001)], 7, 1, 64, 128),
    ([(90, 5000)], 32, 4, 128, 64),
    ([(9, 4000), (2, 300), (33, 40)], 40, 2, 64, 16),  # groups of 20 heads
    ([(140, 150 + 70 * i) for i in range(20)], 4, 2, 64, 64),
    ([(1, 60 + i) for i in range(40)] + [(400, 400)], 16, 2, 128, 16),
]


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_attend_prompts(case, name):
    lens, HQ, HKV, D, page = PROMPTS[case]
    check_attend(attend_problem(name, lens, HQ, HKV, D, page, 60 + case), name)


@pytest.mark.parametrize("causal,window", [(False, -1), (True, 1), (True, 70), (True, 128), (True, 300), (False, 33)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_prompts_masks(causal, window, D):
    lens = [(300, 1000), (129, 129), (1, 400), (200, 170), (80, 1), (66, 0), (400, 700)]
    check_attend(attend_problem("bf16", lens, 6, 2, D, 16, 16, spare_rows=3), "bf16", causal, window)


@pytest.mark.parametrize("causal,window", [(True, -1), (False, -1), (True, 100), (False, 200)])
@pytest.mark.parametrize("lens,HQ,HKV,D,page", [
    ([(65, 65), (128, 128), (70, 129), (100, 256)], 2, 2, 64, 16),           # one block and two
    ([(65, 257), (128, 385), (127, 2000), (66, 66)], 2, 2, 128, 64),
    ([(16, 3000), (9, 128), (13, 513), (16, 16)], 32, 4, 128, 32),           # groups of 8 heads
    ([(70 + i, 200 + 37 * i) for i in range(40)], 12, 12, 64, 64),           # many units a CTA
    ([(80, 300), (300, 400), (90, 1000), (257, 300), (500, 640)], 8, 8, 64, 128),  # beside large ones
    ([(100, 20000)], 1, 1, 128, 128),                                        # many parts of one unit
])
def test_attend_prompts_of_at_most_128_rows(lens, HQ, HKV, D, page, causal, window):
    check_attend(attend_problem("bf16", lens, HQ, HKV, D, page, 80), "bf16", causal, window)


def test_attend_prompts_of_at_most_128_rows_special():
    """Lacking pages, rows without keys, scales far apart, a batch of which one row is not finite."""
    prob = attend_problem("f16", [(100, 700), (90, 20), (70, 0), (128, 900)], 2, 1, 64, 16, 81)
    prob[5][0, 3:30], prob[5][3, :9] = -1, -1
    check_attend(prob, "f16")
    q, kc, vc, ks, vs, table, cu, kv = attend_problem("bf16", [(100, 700), (70, 300)], 2, 1, 128, 32, 82)
    vs = vs * np.exp2(np.random.default_rng(4).integers(-12, 13, vs.shape))
    check_attend((q, kc, vc, ks, vs, table, cu, kv), "bf16")
    ref, rl = run_attend((q, kc, vc, ks, vs, table, cu, kv), "bf16")
    for _ in range(3):
        o, lse = run_attend((q, kc, vc, ks, vs, table, cu, kv), "bf16")
        assert np.array_equal(o, ref) and np.array_equal(lse, rl)
    q[7, 0, 3] = np.nan
    o, lse = run_attend((q, kc, vc, ks, vs, table, cu, kv), "bf16")
    keep = np.ones(o.shape[:2], bool)
    keep[7, 0] = False
    assert np.isnan(o[7, 0]).all() and np.array_equal(o[keep], ref[keep])


def test_attend_prompts_with_lacking_pages_and_far_scales():
    prob = attend_problem("f16", [(200, 900), (120, 500)], 8, 2, 128, 16, 17)
    q, kc, vc, ks, vs, table, cu, kv = prob
    table[0, 3], table[0, 8:25], table[1, :5], table[1, 30] = -1, 1 << 29, -9, -1
    check_attend(prob, "f16")
    rng = np.random.default_rng(5)
    far = (q, kc, vc, ks * np.exp2(rng.integers(-3, 4, ks.shape)), vs * np.exp2(rng.integers(-12, 13, vs.shape)), table,
           cu, kv)
    check_attend(far, "f16", heads_first=True)
    odd = (q, kc, vc, (ks * rng.uniform(0.7, 1.4, ks.shape)).astype(np.float32).astype(np.float64),
           (vs * rng.uniform(0.1, 9.0, vs.shape)).astype(np.float32).astype(np.float64), table, cu, kv)
    check_attend(odd, "f16", v_rounded=True)
    check_attend((q, kc, vc, ks, vs * 0.0, table, cu, kv), "f16")


def test_attend_prompts_of_far_ranges():
    q, kc, vc, ks, vs, table, cu, kv = attend_problem("bf16", [(150, 300), (70, 70)], 4, 1, 64, 16, 18)
    for qs, kz in ((2.0 ** 14, 2.0 ** -14), (2.0 ** -13, 2.0 ** 12)):
        check_attend((q * qs, kc, vc, ks * kz, vs * 2.0 ** 60, table, cu, kv), "bf16")


def test_attend_prompts_not_finite_queries_stay_in_their_rows():
    prob = attend_problem("f16", [(200, 300), (150, 170)], 4, 1, 64, 16, 19)
    ref, rl = run_attend(prob, "f16")
    q = prob[0].copy()
    q[7, 1, 5], q[222, 2, 0] = np.nan, np.inf
    got, gl = run_attend((q,) + prob[1:], "f16")
    bad = np.zeros(gl.shape, bool)
    bad[1, 7] = bad[2, 222] = True
    assert np.isnan(gl[bad]).all() and np.isnan(got[bad.T]).all()
    assert np.array_equal(gl[~bad], rl[~bad]) and np.array_equal(got[~bad.T], ref[~bad.T])


def test_attend_prompts_are_the_same_from_run_to_run():
    prob = attend_problem("bf16", [(700, 3500), (1, 900)], 8, 2, 128, 64, 20)
    a, al = run_attend(prob, "bf16")
    for _ in range(3):
        b, bl = run_attend(prob, "bf16")
        assert np.array_equal(a, b) and np.array_equal(al, bl)


def test_attend_rows_without_keys():
    """No cached token, more queries than keys, no query at all."""
    lens = [(1, 0), (5, 2), (0, 50), (3, 0), (1, 40), (0, 0)]
    for causal in (True, False):
        check_attend(attend_problem("f16", lens, 4, 2, 64, 16, 8, spare_rows=2), "f16", causal)


def test_attend_without_any_query_or_key():
    check_attend(attend_problem("f16", [(0, 5), (0, 0)], 4, 2, 64, 16, 8, spare_rows=4), "f16")
    check_attend(attend_problem("f16", [(2, 0), (1, 0)], 4, 2, 64, 16, 8), "f16")


def test_attend_pages_that_are_lacking():
    prob = attend_problem("bf16", [(1, 500), (2, 333), (1, 48)], 8, 2, 128, 16, 9)
    table = prob[5]
    table[0, 3], table[0, 30], table[1, :5], table[2, :3] = -1, 1 << 29, -9, -1
    check_attend(prob, "bf16")


def test_attend_past_the_table():
    """Lengths past the table's width: what the table cannot hold is not seen."""
    q, kc, vc, ks, vs, table, cu, kv = attend_problem("f16", [(1, 64), (3, 40)], 4, 2, 64, 16, 10)
    check_attend((q, kc, vc, ks, vs, table[:, :4].copy(), cu, kv + [5, 0]), "f16")
    check_attend((q, kc, vc, ks, vs, table[:, :4].copy(), cu, kv + [2 ** 31 - 65, 0]), "f16", causal=False)


@pytest.mark.parametrize("m", [1, 40])
def test_attend_pages_held_twice(m):
    """A prefix that two requests share, and a page twice in one row."""
    q, kc, vc, ks, vs, table, cu, kv = attend_problem("bf16", [(m, 200), (m + 1, 180), (m, 300)], 8, 2, 64, 32, 30)
    table[1, :4] = table[0, :4]
    table[2, 5] = table[2, 2]
    table[2, 7] = table[1, 1]
    check_attend((q, kc, vc, ks, vs, table, cu, kv), "bf16")


def test_attend_of_other_layouts_and_scales():
    prob = attend_problem("bf16", [(1, 700), (3, 90)], 8, 2, 128, 64, 11, size=0.1)
    check_attend(prob, "bf16", scale=0.3, heads_first=True)
    q, kc, vc, ks, vs, table, cu, kv = prob
    # any positive scales, far apart
    rng = np.random.default_rng(3)
    ks = (ks * rng.uniform(0.7, 1.4, ks.shape)).astype(np.float32).astype(np.float64)
    vs = (vs * rng.uniform(0.1, 9.0, vs.shape)).astype(np.float32).astype(np.float64)
    check_attend((q, kc, vc, ks, vs, table, cu, kv), "bf16")


@pytest.mark.parametrize("qs,ksz", [(2.0 ** 14, 2.0 ** -14), (2.0 ** -13, 2.0 ** 12)])
def test_attend_of_far_ranges(qs, ksz):
    """Queries and cached values at the ends of their ranges."""
    q, kc, vc, ks, vs, table, cu, kv = attend_problem("bf16", [(1, 300), (2, 50)], 4, 1, 64, 16, 12)
    check_attend((q * qs, kc, vc, ks * ksz, vs * 2.0 ** 60, table, cu, kv), "bf16")
    check_attend((q * qs, kc, vc, ks * ksz, vs * 0.0, table, cu, kv), "bf16")


def test_attend_of_not_finite_queries_stays_in_its_row():
    prob = attend_problem("f16", [(1, 200), (2, 90)], 4, 1, 64, 16, 13)
    ref, rl = run_attend(prob, "f16")
    q = prob[0].copy()
    q[0, 1, 5], q[2, 2, 0] = np.nan, np.inf
    got, gl = run_attend((q,) + prob[1:], "f16")
    bad = np.zeros(gl.shape, bool)
    bad[1, 0] = bad[2, 2] = True
    assert np.isnan(gl[bad]).all() and np.isnan(got[bad.T]).all()
    assert np.array_equal(gl[~bad], rl[~bad]) and np.array_equal(got[~bad.T], ref[~bad.T])


def test_attend_strided_queries_and_outputs():
    import torch

    import attention_backward_gb300 as ab

    prob = attend_problem("bf16", [(1, 300), (4, 70)], 8, 2, 64, 16, 14)
    q, kc, vc, ks, vs, table, cu, kv = prob
    ref, rl = run_attend(prob, "bf16")
    qkv = torch.full((1, 5, 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, :, :8] = cuda(q, torch.bfloat16)
    wide = torch.full((1, 5, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = wide[:, :, 1:, 64:], torch.empty(1, 5, 8, device="cuda").transpose(1, 2)
    tab = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    tab[:, :table.shape[1]] = i32(table)
    ab.forward_kv_cache(qkv[:, :, :8], fp8(kc), fp8(vc), cuda(ks.astype(np.float32)), cuda(vs.astype(np.float32)),
                        tab[:, :table.shape[1]], i32(cu), i32(kv), out=(o, lse))
    assert np.array_equal(o[0].double().cpu().numpy(), ref) and np.array_equal(lse[0].double().cpu().numpy(), rl)
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, :, :64] == 7).all()


def test_attend_is_the_same_from_run_to_run():
    prob = attend_problem("f16", [(1, 6000), (3, 2500), (1, 20)], 16, 2, 128, 64, 15)
    a, al = run_attend(prob, "f16")
    for _ in range(3):
        b, bl = run_attend(prob, "f16")
        assert np.array_equal(a, b) and np.array_equal(al, bl)


# ------------------------------------------------------------------ together


class Server:
    """A few requests served from one cache, the host keeping f64 copies."""

    def __init__(self, name, n, HQ, HKV, D, page, blocks, seed):
        import torch

        import attention_backward_gb300 as ab

        self.ab, self.name, self.rng = ab, name, np.random.default_rng(seed)
        self.n, self.HQ, self.HKV, self.D, self.page, self.nb = n, HQ, HKV, D, page, blocks
        self.cache = ab.new_kv_cache(blocks, page, HKV, D)
        self.table = torch.full((n, blocks), -1, dtype=torch.int32, device="cuda")
        self.free = i32(self.rng.permutation(blocks))
        self.start = i32([0])
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")

    def inputs(self, T):
        return [cuda(rounded(self.rng, (1, T, h, self.D), self.name), dt_of(self.name))
                for h in (self.HQ, self.HKV, self.HKV)]

    def step(self, new, q, k, v, T, out=None, plan=None, window=-1):
        ab = self.ab
        plan = ab.kv_block_tables(self.lens, new, self.table, self.free, self.page, self.nb, T, self.start, plan)
        ab.kv_cache_write(k, v, plan.slot_map, *self.cache)
        o = ab.forward_kv_cache(q, *self.cache, self.table, plan.cu_seqlens, plan.kv_lens, window=window, out=out)
        self.start += plan.counts[1:2]
        self.lens.copy_(plan.kv_lens)
        return plan, o

    def check(self, plan, q, o, lse, window=-1):
        """O and LSE against the oracle on the cache's present contents."""
        kc, vc, ks, vs = self.cache
        T = int(plan.cu_seqlens[-1])
        prob = (q[0].double().cpu().numpy(), bytes_of(kc), bytes_of(vc), ks.double().cpu().numpy(),
                vs.double().cpu().numpy(), self.table.cpu().numpy(), plan.cu_seqlens.cpu().numpy(),
                plan.kv_lens.cpu().numpy())
        ro, rl, mag, dots, seen, vmax = oracle.forward(*prob, self.D ** -0.5, True, window)
        half = 2.0 ** -11 if self.name == "f16" else 2.0 ** -8
        e = 2 * (self.D * 2.0 ** -23 * dots + 2.0 ** -21)
        tol = half * np.abs(ro) + (2.0 ** -11 + e.T[..., None]) * mag * (1 + half) + \
            (2.0 ** -24 * seen * vmax).T[..., None] + 2.0 ** -25
        assert (np.abs(o[0].double().cpu().numpy() - ro)[:T] <= tol[:T]).all()
        assert np.abs(lse[0].double().cpu().numpy() - rl)[:, :T].max() <= e.max() + 1e-5


@pytest.mark.parametrize("name,D,page,window", [("bf16", 128, 16, -1), ("f16", 64, 64, 50)])
def test_prompts_then_tokens(name, D, page, window):
    """Prompts, drafted tokens and single tokens served step after step; the
    cache holds every key and value within half an e4m3 step of its page."""
    s = Server(name, 3, 8, 2, D, page, 64, 21)
    keys = [[] for _ in range(3)]
    for new in ([130, 1, 70], [1, 1, 1], [4, 0, 2], [1, 1, 1], [0, 90, 1]):
        T = sum(new)
        q, k, v = s.inputs(T)
        plan, (o, lse) = s.step(i32(new), q, k, v, T, window=window)
        assert plan.counts[2].item() == 0
        s.check(plan, q, o, lse, window)
        at = 0
        for r, m in enumerate(new):
            keys[r].append(k[0, at:at + m].double().cpu().numpy())
            at += m
    kc, ks = bytes_of(s.cache[0]), s.cache[2].double().cpu().numpy()
    table = s.table.cpu().numpy()
    for r in range(3):
        x = np.concatenate(keys[r])
        assert s.lens[r].item() == len(x)
        pos = np.arange(len(x))
        blk = table[r, pos // page]
        y = oracle.E4M3[kc[blk, pos % page]] * ks[blk][:, :, None]
        # half a step of 2^-3 relative, and of 2^-9 times the scale; a page's
        # scale may have been raised after its first tokens (another such step)
        assert (np.abs(y - x) <= 2.0 ** -4 * np.abs(x) + 2 * 2.0 ** -10 * ks[blk][:, :, None]).all()
    assert len(np.unique(table[table >= 0])) == (table >= 0).sum()  # no page is held twice


def test_step_captured_and_replayed():
    """One captured step, replayed while the lengths grow on the device; two
    graphs that share a workspace and outputs run one after the other."""
    import torch

    import attention_backward_gb300 as ab

    s = Server("bf16", 4, 8, 2, 64, 16, 200, 22)
    q, k, v = s.inputs(40)
    s.step(i32([20, 3, 16, 1]), q, k, v, 40)
    T = 6  # room for six new tokens a step
    q, k, v = s.inputs(T)
    new = i32([1, 1, 1, 1])
    plan = ab.KvPlan(*(torch.empty(m, dtype=torch.int32, device="cuda") for m in (5, 4, T, T, 3)))
    out = (torch.empty_like(q), torch.empty(1, 8, T, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    start, lens, table = s.start.clone(), s.lens.clone(), s.table.clone()
    with torch.cuda.stream(side):
        s.step(new, q, k, v, T, out, plan)
    torch.cuda.synchronize()
    s.start.copy_(start), s.lens.copy_(lens), s.table.copy_(table)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            s.step(new, q, k, v, T, out, plan)
    assert torch.equal(s.lens, lens)  # capturing runs nothing
    steps = [[1, 1, 1, 1], [3, 0, 1, 2], [0, 0, 0, 1], [1, 2, 1, 1], [1, 1, 1, 1]] * 3
    for i, m in enumerate(steps):
        for t in (q, k, v):
            t.copy_(cuda(rounded(s.rng, tuple(t.shape), "bf16"), torch.bfloat16))
        new.copy_(i32(m))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert plan.counts.tolist()[0] == sum(m) and plan.counts[2].item() == 0
        s.check(plan, q, out[0], out[1])
    assert s.lens.tolist() == (np.array([20, 3, 16, 1]) + np.array(steps).sum(0)).tolist()


def test_calls_on_another_stream():
    import torch

    import attention_backward_gb300 as ab

    prob = attend_problem("bf16", [(1, 900), (2, 100)], 8, 2, 64, 16, 23)
    ref, rl = run_attend(prob, "bf16")
    q, kc, vc, ks, vs, table, cu, kv = prob
    args = (cuda(q, torch.bfloat16)[None], fp8(kc), fp8(vc), cuda(ks.astype(np.float32)), cuda(vs.astype(np.float32)),
            i32(table), i32(cu), i32(kv))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        outs = [ab.forward_kv_cache(*args, stream=stream) for _ in range(4)]
        side.synchronize()
        for o, lse in outs:
            assert np.array_equal(o[0].double().cpu().numpy(), ref)
            assert np.array_equal(lse[0].double().cpu().numpy(), rl)


def test_two_streams_with_workspaces_of_their_own():
    import torch

    import attention_backward_gb300 as ab

    prob = attend_problem("f16", [(1, 3000), (1, 50)], 8, 2, 128, 64, 24)
    ref, rl = run_attend(prob, "f16")
    q, kc, vc, ks, vs, table, cu, kv = prob
    args = (cuda(q, torch.float16)[None], fp8(kc), fp8(vc), cuda(ks.astype(np.float32)), cuda(vs.astype(np.float32)),
            i32(table), i32(cu), i32(kv))
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(2)] * 5:
        got.append(ab.forward_kv_cache(*args, stream=s))
    torch.cuda.synchronize()
    for o, lse in got:
        assert np.array_equal(o[0].double().cpu().numpy(), ref) and np.array_equal(lse[0].double().cpu().numpy(), rl)


def test_prompt_graphs_side_by_side():
    """Mixed batches captured with a workspace each, replayed at the same time
    on two streams and again with other lengths in the same buffers."""
    import torch

    import attention_backward_gb300 as ab

    probs = [attend_problem("bf16", lens, 16, 2, 128, 64, 31 + i)
             for i, lens in enumerate([[(300, 900), (1, 700), (3, 64)], [(2, 500), (1, 900), (301, 400)]])]
    refs = [run_attend(p, "bf16") for p in probs]
    assert probs[0][0].shape == probs[1][0].shape
    sides, graphs, held = [torch.cuda.Stream() for _ in range(2)], [], []
    for (q, kc, vc, ks, vs, table, cu, kv), st in zip(probs, sides):
        args = [cuda(q, torch.bfloat16)[None], fp8(kc), fp8(vc), cuda(ks.astype(np.float32)),
                cuda(vs.astype(np.float32)), i32(table), i32(cu), i32(kv)]
        ws = torch.empty(ab.kv_cache_workspace_size(q.shape[0], 16, 2, 128), dtype=torch.uint8, device="cuda")
        out = (torch.empty_like(args[0]), torch.empty(1, 16, q.shape[0], device="cuda"))
        ab.forward_kv_cache(*args, workspace=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            ab.forward_kv_cache(*args, workspace=ws, out=out)
        graphs.append(g)
        held.append((args, ws, out))
    for _ in range(5):
        for _, _, out in held:
            out[0].fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, sides):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for (_, _, (o, lse)), (ref, rl) in zip(held, refs):
            assert np.array_equal(o[0].double().cpu().numpy(), ref)
            assert np.array_equal(lse[0].double().cpu().numpy(), rl)
    # the second batch's row ranges and lengths in the first graph's buffers
    (args, ws, out), (_, kc, vc, ks, vs, table, cu, kv) = held[0], probs[0]
    cu, kv = probs[1][6], np.array([400, 650, 64])
    args[6].copy_(i32(cu)), args[7].copy_(i32(kv))
    graphs[0].replay()
    torch.cuda.synchronize()
    ref, rl = run_attend((probs[0][0], kc, vc, ks, vs, table, cu, kv), "bf16")
    assert np.array_equal(out[0][0].double().cpu().numpy(), ref)
    assert np.array_equal(out[1][0].double().cpu().numpy(), rl)
    check_attend((probs[0][0], kc, vc, ks, vs, table, cu, kv), "bf16")


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 33, 70]])
def test_offsets_past_32_bits(new):
    """Pages beyond 4 GB of the caches, rows of q and o beyond 4 GB: the same
    results, bit for bit, as from small buffers."""
    import torch

    import attention_backward_gb300 as ab

    HQ, HKV, D, page = 8, 4, 128, 16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    ctx, T = [50, 0, 33], sum(new)
    rng = np.random.default_rng(90)
    lens = np.array(ctx) + new
    width = int(-(-lens.max() // page)) + 1
    small = np.arange(3 * width).reshape(3, width)
    nb = (1 << 32) // (page * HKV * D) + 4000
    x = [cuda(rounded(rng, (1, int(lens.sum()), HKV, D), "bf16"), torch.bfloat16) for _ in range(2)]
    q = cuda(rounded(rng, (1, T, HQ, D), "bf16"), torch.bfloat16)
    wide = (2 ** 31 // (T - 1) // 8 + 1) * 8  # elements between rows: the last one lies past 2^32 bytes
    results = []
    for big in (False, True):
        table = nb - 1 - 7 * small if big else small
        caches = [torch.empty(nb if big else 3 * width, page, HKV, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        caches = [c.view(torch.float8_e4m3fn) for c in caches]
        scales = [torch.zeros(c.shape[0], HKV, device="cuda") for c in caches]
        slots = np.concatenate([table[r, np.arange(n) // page] * page + np.arange(n) % page for r, n in enumerate(lens)])
        assert not big or slots.min() * HKV * D > 2 ** 32
        ab.kv_cache_write(x[0], x[1], i32(slots), *caches, *scales)
        tq, o = q, torch.zeros_like(q)
        if big:
            room = torch.empty(2, T * wide, dtype=torch.bfloat16, device="cuda")
            tq, o = (r.as_strided((1, T, HQ, D), (T * wide, wide, D, 1), r.storage_offset()) for r in room)
            tq.copy_(q)
        lse = torch.zeros(1, HQ, T, device="cuda")
        cu = np.concatenate([[0], np.cumsum(new)])
        ab.forward_kv_cache(tq, *caches, *scales, i32(table), i32(cu), i32(lens), out=(o, lse))
        torch.cuda.synchronize()
        results.append((o.clone(), lse.clone()))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert results[0][0].abs().max() > 0.1


def test_no_tokens():
    import torch

    import attention_backward_gb300 as ab

    kc, vc, ks, vs = ab.new_kv_cache(4, 16, 2, 64)
    e = torch.empty(1, 0, 2, 64, dtype=torch.float16, device="cuda")
    ab.kv_cache_write(e, e, i32(np.zeros(0)), kc, vc, ks, vs)
    o, lse = ab.forward_kv_cache(e, kc, vc, ks, vs, i32([[0, 1]]), i32([0, 0]), i32([5]))
    assert o.shape == (1, 0, 2, 64) and lse.shape == (1, 2, 0)
    plan = ab.kv_block_tables(i32([5]), i32([0]), i32([[0, -1]]), i32([1, 2]), 16, 4, 0)
    assert plan.counts.tolist() == [0, 0, 0] and plan.kv_lens.tolist() == [5]
