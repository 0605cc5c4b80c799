"""Attention over the 8-bit cache where V scales of a head lie far apart, against
a plain form in 64 bits.

A query's weights are p_j, its softmax, times vs_j, the V scale of the key's page.
The kernels round p_j vs_j to fp16 after a power of two of the row's own, which
keeps the row's largest p_j vs_j above half of 2^top when it is set.  Below fp16's
normal range a rounding is off by at most half its smallest step, 2^-25, so the
bound of O, element by element, is
  eps/2 |o|                                 the rounding of the output
  2^-11 sum p |v|                           fp16 rounding of the weights
  sum p e |v| + |o| sum p e                 errors e_j of their exponents, in the
                                            numerator and the denominator
  2^-25 / 2^(top - 1) max_j p_j vs_j sum b  weights below fp16's normal range, b the
                                            absolute values that the bytes of the seen keys stand for
with e_j = D 2^-23 sum |q||k_j| scale + 2^-21: f32 sums of D products, the rounding
of the scaled score and of its power.  The LSE has sum p e + 2^-23 |lse| + 2^-20.
Nothing of a key that the row does not see enters.  ``top``: FEW_TOP for the kernel of few rows, MANY_TOP
for that of many (kv_decode.cu, kv_prompt.cu).
"""
import numpy as np
import pytest

from oracle import kv_cache as oracle
from test_gpu_kv_cache import attend_problem, rounded, run_attend

pytestmark = pytest.mark.gpu

FEW_TOP, MANY_TOP = 7, 3


def plain(prob, causal, window, scale):
    """Row by row: O, sum p |v|, the error of O by the exponents, LSE and its
    error, the largest p vs times the sums of the bytes' values.  Rows of no key have O = 0."""
    q, kc, vc, ks, vs, table, cu, kv = prob
    T, HQ, D = q.shape
    page, HKV = kc.shape[1], kc.shape[2]
    o, mag, oe, low = (np.zeros((T, HQ, D)) for _ in range(4))
    lse, le = np.full((T, HQ), -np.inf), np.zeros((T, HQ))
    for n, L in enumerate(kv):
        m = cu[n + 1] - cu[n]
        for i in range(m):
            at = L - m + i
            j = np.arange(max(0, at - window + 1) if window > 0 else 0, at + 1 if causal or window > 0 else L)
            if len(j) == 0:
                continue
            blk, t = table[n, j // page], cu[n] + i
            for f in range(HQ):
                h = f * HKV // HQ
                K = oracle.E4M3[kc[blk, j % page, h]] * ks[blk, h][:, None]
                b = oracle.E4M3[vc[blk, j % page, h]]
                V = b * vs[blk, h][:, None]
                x = K @ q[t, f] * scale
                p = np.exp(x - x.max())
                lse[t, f] = x.max() + np.log(p.sum())
                p /= p.sum()
                e = D * 2.0 ** -23 * (np.abs(K) @ np.abs(q[t, f])) * scale + 2.0 ** -21
                o[t, f], mag[t, f], le[t, f] = p @ V, p @ np.abs(V), p @ e
                oe[t, f] = (p * e) @ np.abs(V) + np.abs(o[t, f]) * le[t, f]
                low[t, f] = (p * vs[blk, h]).max() * np.abs(b).sum(0)
    return o, mag, oe, lse, le, low


def check(prob, name, causal=True, window=-1, top=0):
    scale = prob[0].shape[2] ** -0.5
    got, glse = run_attend(prob, name, causal, window)
    o, mag, oe, lse, le, low = plain(prob, causal, window, scale)
    none = np.isneginf(lse)
    assert (got[none] == 0).all() and np.isneginf(glse.T[none]).all()
    el, tl = np.abs(glse.T - lse)[~none], (le + 2.0 ** -23 * np.abs(lse) + 2.0 ** -20)[~none]
    assert (el <= tl).all(), (el / tl).max()
    half, tiny = (2.0 ** -11, 2.0 ** -25) if name == "f16" else (2.0 ** -8, 0.0)
    tol = half * np.abs(o) + (2.0 ** -11 * mag + oe + 2.0 ** (-24 - top) * low) * (1 + half) + tiny
    err = np.abs(got - o)
    assert np.isfinite(got).all() and (err <= tol).all(), (err / np.where(tol > 0, tol, 1)).max()


def pages_of(prob, n, first, last):
    """Pages of request n that hold its positions [first, last)."""
    page = prob[1].shape[1]
    return prob[5][n, first // page:-(-last // page)]


FEW = [([(6, 66)], 2, 2, 64, 16), ([(4, 1026)], 8, 2, 128, 64), ([(3, 2050), (1, 40), (2, 130)], 6, 1, 128, 128)]
MANY = [([(150, 200)], 2, 1, 64, 16), ([(300, 700)], 4, 4, 128, 64), ([(90, 5000), (70, 90)], 2, 1, 64, 32)]


@pytest.mark.parametrize("up", [2.0 ** 26, 1.3 * 2.0 ** 24, 2.0 ** 40])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_rows_beside_a_page_that_some_do_not_see(case, up):
    """A page's V scale is far above the others'.  The last page, before which the
    first queries end; then one that the windows of the last queries begin behind."""
    lens, HQ, HKV, D, page = FEW[case]
    m, L = lens[0]
    assert L % page < m
    prob = attend_problem("bf16", lens, HQ, HKV, D, page, 200 + case)
    prob[4][pages_of(prob, 0, L // page * page, L)] *= np.float32(up)
    check(prob, "bf16")
    prob = attend_problem("bf16", lens, HQ, HKV, D, page, 200 + case)
    begin = (L - m) // page * page
    prob[4][pages_of(prob, 0, begin - page, begin)] *= np.float32(up)
    check(prob, "bf16", window=L - begin - m // 2)


@pytest.mark.parametrize("up", [2.0 ** 26, 1.3 * 2.0 ** 24, 2.0 ** 40])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows_beside_pages_that_some_do_not_see(case, up):
    lens, HQ, HKV, D, page = MANY[case]
    prob = attend_problem("bf16", lens, HQ, HKV, D, page, 210 + case)
    m, L = lens[0]
    prob[4][pages_of(prob, 0, L - m // 2, L)] *= np.float32(up)
    check(prob, "bf16")


def against(prob, n, first, last, size):
    """Keys [first, last) of request n point against its queries' mean (size < 0) or
    along it (size > 0): scores of about ``size`` where the queries are one.
    (Their pages' K scales change: whole pages, but for the test of one key.)"""
    q, kc, _, ks, _, table, cu, _ = prob
    page, HKV = kc.shape[1], kc.shape[2]
    rows = q[cu[n]:cu[n + 1]]
    g = rows.shape[1] // HKV
    for h in range(HKV):
        d = rows[:, h * g:(h + 1) * g].mean((0, 1))
        d = d / (d @ d) * size * q.shape[2] ** 0.5
        for j in range(first, last):
            b = table[n, j // page]
            ks[b, h] = 2.0 ** -3
            kc[b, j % page, h] = oracle.to_e4m3(d / ks[b, h])


@pytest.mark.parametrize("page,up", [(16, 2.0 ** 16), (64, 2.0 ** 20), (32, 1.7 * 2.0 ** 25)])
@pytest.mark.parametrize("lens,HQ,D", [([(1, 900)], 2, 64), ([(1, 5000), (1, 700)], 1, 128), ([(100, 1000)], 1, 128)])
def test_a_far_larger_page_of_no_weight(lens, HQ, D, page, up):
    """Scores of 100 below the others': its V scale says nothing about the row."""
    prob = attend_problem("f16", lens, HQ, HQ, D, page, 220 + page)
    rng = np.random.default_rng(5)
    prob[0][:] = rounded(rng, (1, HQ, D), "f16")  # the same query in all rows: one direction is against them all
    for n in range(len(lens)):
        against(prob, n, 2 * page, 3 * page, -100)
        prob[4][pages_of(prob, n, 2 * page, 3 * page)] *= np.float32(up)
    check(prob, "f16")


@pytest.mark.parametrize("vs", [0.0, 2.0 ** -100])
@pytest.mark.parametrize("at", [0, 3])
@pytest.mark.parametrize("lens,HQ,D", [([(1, 900)], 2, 64), ([(1, 5000)], 1, 128), ([(100, 1000)], 1, 64)])
def test_a_page_of_zeros_with_the_weight(lens, HQ, D, at, vs):
    """A page of zero values far above the others in score (a sink), met first or
    later: what little the others weigh is all there is of O."""
    prob = attend_problem("bf16", lens, HQ, HQ, D, 16, 230)
    prob[0][:] = rounded(np.random.default_rng(6), (1, HQ, D), "bf16")
    against(prob, 0, at * 16, at * 16 + 16, 18)
    blk = prob[5][0, at]
    prob[2][blk], prob[4][blk] = 0, vs
    check(prob, "bf16")


@pytest.mark.parametrize("lens", [[(1, 3000), (5, 77)], [(120, 600)]])
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_scales_of_any_size(name, lens):
    """V scales of the pages spread over 2^60, no powers of two; some are zero."""
    prob = attend_problem(name, lens, 4, 2, 64, 16, 240)
    rng = np.random.default_rng(7)
    vs = prob[4] * np.exp2(rng.uniform(-45, 6, prob[4].shape))
    vs[rng.random(vs.shape) < 0.2] = 0
    prob = prob[:4] + (vs.astype(np.float32).astype(np.float64),) + prob[5:]
    check(prob, name)
    check(prob, name, window=20)
    check(prob, name, causal=False)


@pytest.mark.parametrize("lens,HQ,D", [([(1, 900)], 2, 64), ([(1, 40000)], 1, 128), ([(1, 5000), (1, 700)], 2, 128),
                                       ([(100, 1000)], 1, 64), ([(80, 5000)], 1, 128)])
@pytest.mark.parametrize("size", [14, 17, 18])
def test_one_key_with_the_weight(lens, HQ, D, size):
    """A key without value far above the others in score: weights of 2^-20, 2^-24.5
    and 2^-26 of its own are all there is of O.  The others' scores are equal and
    their values of one sign, so that what is lost of them adds up."""
    prob = attend_problem("bf16", lens, HQ, HQ, D, 16, 250)
    q, kc, vc, ks, vs, table, cu, kv = prob
    q[:] = rounded(np.random.default_rng(8), (1, HQ, D), "bf16")
    for n, L in enumerate(kv):
        j = np.arange(L)
        kc[table[n, j // 16], j % 16] = 0
        vc[table[n, j // 16], j % 16] &= 0x7F
        vs[table[n, j // 16]] = 2.0 ** -6
        against(prob, n, 0, 1, size)
        vc[table[n, 0], 0] = 0
    check(prob, "bf16", top=FEW_TOP if lens[0][0] == 1 else MANY_TOP)


@pytest.mark.parametrize("lens", [[(1, 3000), (5, 77)], [(120, 600), (70, 90)]])
def test_rows_of_the_smallest_scales_alone(lens):
    """Pages at a write's smallest scale, 2^-100, that some rows see alone and others
    beside ordinary ones; their largest weights sit at 1."""
    prob = attend_problem("bf16", lens, 4, 2, 64, 16, 260)
    kv, vs = prob[7], prob[4]
    for n, L in enumerate(kv):
        vs[pages_of(prob, n, 0, L - (lens[n][0] + 1) // 2)] = 2.0 ** -100
    check(prob, "bf16", top=0)
    check(prob, "bf16", window=20, top=0)


@pytest.mark.parametrize("lens", [[(1, 9000), (5, 77)], [(120, 4000), (70, 90)]])
def test_scales_up_to_the_largest(lens):
    """2^70, on rows whose keys are split over workers too, alone and beside ordinary pages."""
    prob = attend_problem("bf16", lens, 4, 2, 64, 16, 270)
    q, kc, vc, ks, vs, table, cu, kv = prob
    check((q, kc, vc, ks, vs * 2.0 ** 75, table, cu, kv), "bf16", top=0)
    rng = np.random.default_rng(9)
    some = vs * np.where(rng.random(vs.shape) < 0.3, 2.0 ** 75, 1.0)
    check((q, kc, vc, ks, some, table, cu, kv), "bf16", window=100, top=0)
