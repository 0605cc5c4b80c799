"""GPU parity of rotary positions and the latent cache write with their float64
definitions.

Tolerance of a turned value y = s (x1 cos t -+ x2 sin t), element by element: eps/2 |y|
for its rounding, 2^-20 s (|x1| + |x2|) for the f32 angle, cosine, sine, products and sum
(a few steps of 2^-24 each; the angle's fixed point adds 1.5e-9), and half the type's
smallest step.  A normalised one: eps/2 |y| + 2^-20 |y| and half the smallest step (sums
of 512 squares of one sign are within 2^-19.8 in the worst order and enter under a root).
"""
import numpy as np
import pytest

from oracle import latent as oracle

pytestmark = pytest.mark.gpu

EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
STEP = {"f16": 2.0 ** -25, "bf16": 0.0}


def dt_of(name):
    import torch

    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def rounded(rng, shape, name, size=1.0):
    """Normal values of a 16-bit type on the GPU."""
    import torch

    return torch.from_numpy(rng.standard_normal(shape) * size).to(dt_of(name)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def i32(x):
    import torch

    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def near(got, y, size, name):
    tol = EPS[name] * np.abs(y) + 2.0 ** -20 * size + STEP[name]
    err = np.abs(f64(got) - y)
    assert (err <= tol).all(), (err / tol).max()


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0, base=500000.0),
            dict(scaling="parts", factor=32.0, original_length=4096)]


@pytest.mark.parametrize("B,S,HQ,HK,DQ,DK,R,sq,sk,name,inter,inverse", [
    (1, 1, 1, 0, 16, 0, 16, 0, 0, "bf16", False, False), (3, 5, 32, 8, 128, 128, 128, 0, 0, "bf16", False, False),
    (2, 37, 7, 1, 192, 64, 64, 128, 0, "f16", True, False), (1, 130, 64, 1, 576, 576, 64, 512, 512, "bf16", True, True),
    (1, 3, 5, 5, 104, 136, 96, 8, 16, "f16", False, True), (2, 600, 33, 4, 72, 64, 32, 24, 8, "f16", True, False),
    (1, 2000, 130, 9, 128, 128, 128, 0, 0, "bf16", False, True), (64, 1, 20, 2, 64, 64, 64, 0, 0, "f16", False, False)])
def test_rope(B, S, HQ, HK, DQ, DK, R, sq, sk, name, inter, inverse):
    import attention_backward_gb300 as ab

    rng = np.random.default_rng(B * 1000 + S)
    kw = SCALINGS[(S + HQ) % 4]
    table = ab.rope_table(R, **kw)
    freqs, scale = ab.rope_frequencies(R, **kw)
    q = rounded(rng, (B, S, HQ, DQ), name)
    k = rounded(rng, (B, S, HK, DK), name) if HK else None
    pos = rng.integers(-5, 1000000, (B, 1)) + np.arange(S)
    yq, yk = ab.rope(q, i32(pos), table, k=k, interleaved=inter, start=sq, k_start=sk, inverse=inverse)
    for x, y, start in ((q, yq, sq), (k, yk, sk)):
        if x is None:
            assert y is None
            continue
        ref, size = oracle.turn(f64(x), start, freqs, pos[:, :, None], scale, inter, inverse)
        near(y, ref, scale * size, name)
        rest = [c for c in range(x.shape[3]) if not start <= c < start + R]
        assert (y[..., rest] == x[..., rest]).all()
    # in place, the other columns untouched (NaN among them)
    x = q.clone()
    rest = [c for c in range(DQ) if not sq <= c < sq + R]
    x[..., rest] = float("nan")
    z, _ = ab.rope(x, i32(pos), table, interleaved=inter, start=sq, inverse=inverse, out=(x, None))
    assert z is x and (x[..., sq:sq + R] == yq[..., sq:sq + R]).all() and x[..., rest].isnan().all()


def test_rope_strided_views_and_shared_positions():
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(4)
    both = rounded(rng, (2, 9, 14, 80), "bf16")  # heads of q and k in one projection
    q, k = both[:, :, :10], both[:, :, 10:]
    pos = i32(rng.integers(0, 5000, 9))
    table = ab.rope_table(64, base=1e6)
    yq, yk = ab.rope(q, pos, table, k=k, start=16, k_start=8)
    one, _ = ab.rope(q.contiguous(), pos[None].expand(2, 9).contiguous(), table, start=16)
    assert torch.equal(yq, one)
    out = torch.full((9, 2, 4, 80), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)  # sequence first
    ab.rope(k, pos, table, start=8, out=(out, None))
    assert torch.equal(out, yk)
    empty, _ = ab.rope(q[:, :0], pos[:0], table)
    assert empty.shape == (2, 0, 10, 80)


def test_rope_inverse_is_the_gradient():
    """sum(dy . rope(x)) has the gradient rope(dy, inverse): <dy, rope(x)> =
    <rope^-1(dy), x> for one-hot x, which a column of the map is, within the values'
    roundings; and a turn there and back gives x."""
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(5)
    table = ab.rope_table(32, scaling="parts", factor=16.0, original_length=512)
    pos = i32([70001])
    for inter in (False, True):
        eye = torch.eye(32, dtype=torch.float16, device="cuda")[None, None]  # heads: one-hot columns
        m, _ = ab.rope(eye, pos, table, interleaved=inter)
        t, _ = ab.rope(eye, pos, table, interleaved=inter, inverse=True)
        assert (m[0, 0].float() - t[0, 0].float().t()).abs().max() <= 2.0 ** -20
        # differences of the f64 map agree with the kernel's gradient
        dy = rounded(rng, (1, 1, 1, 32), "f16")
        dx, _ = ab.rope(dy, pos, table, interleaved=inter, inverse=True)
        freqs, scale = ab.rope_frequencies(32, scaling="parts", factor=16.0, original_length=512)
        x = rng.standard_normal((1, 1, 1, 32))
        for c in range(32):
            up, down = x.copy(), x.copy()
            up[..., c] += 0.5
            down[..., c] -= 0.5
            f = [oracle.turn(z, 0, freqs, 70001, scale, inter)[0] for z in (up, down)]
            want = ((f[0] - f[1]) * f64(dy)).sum()
            assert abs(float(dx[0, 0, 0, c]) - want) <= EPS["f16"] * abs(want) + 2.0 ** -20 * 8 + STEP["f16"]


def test_rope_on_another_stream_and_captured():
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(6)
    table = ab.rope_table(64)
    q, k = rounded(rng, (1, 50, 4, 64), "bf16"), rounded(rng, (1, 50, 2, 64), "bf16")
    pos = i32(np.arange(50))
    want = ab.rope(q, pos, table, k=k)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = ab.rope(q, pos, table, k=k, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = (torch.empty_like(q), torch.empty_like(k))
    ab.rope(q, pos, table, k=k, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ab.rope(q, pos, table, k=k, out=out)
    pos += 1000
    graph.replay()
    later = ab.rope(q, pos, table, k=k)
    assert all(torch.equal(a, b) for a, b in zip(out, later)) and not torch.equal(out[0], want[0])


@pytest.mark.parametrize("T,page,name,norm,inter,turns,out", [
    (1, 16, "bf16", True, True, True, None), (2, 64, "f16", False, False, True, "new"), (7, 32, "bf16", True, False, False, "same"),
    (300, 128, "f16", True, True, True, "same"), (1031, 16, "bf16", False, False, False, None),
    (4099, 64, "bf16", True, False, True, "new")])
def test_latent_cache_write(T, page, name, norm, inter, turns, out):
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(T)
    nb = T // page + 3
    kv = rounded(rng, (1, T, 576), name, size=3.0)
    weight = rounded(rng, (512,), name) if norm else None
    slots = rng.permutation(nb * page)[:T]
    skip = rng.random(T) < 0.2
    skip[0] = False
    slots[skip] = rng.choice([-1, nb * page, 2 ** 31 - 1, -2 ** 31], skip.sum())
    pos = rng.integers(0, 200000, T)
    cache = ab.new_latent_cache(nb, page, dt_of(name))
    cache.fill_(11.0)
    kw = dict(base=50000.0, scaling="linear", factor=2.0)
    freqs = ab.rope_frequencies(64, **kw)[0] if turns else None
    x = f64(kv)[0]
    dst = None if out is None else kv if out == "same" else torch.empty_like(kv)
    ab.latent_cache_write(kv, i32(slots), cache, norm_weight=weight, norm_eps=1e-5,
                          positions=i32(pos) if turns else None, table=ab.rope_table(64, scale=1.25, **kw) if turns else None,
                          interleaved=inter, out=dst)
    ref, size = oracle.cache_rows(x, None if weight is None else f64(weight), 1e-5, freqs, pos, 1.25, inter)
    rows = cache.view(-1, 576)
    live = np.flatnonzero(~skip)
    near(rows[torch.from_numpy(slots[live]).cuda()], ref[live], size[live], name)
    other = np.ones(nb * page, bool)
    other[slots[live]] = False
    assert (rows[torch.from_numpy(other).cuda()] == 11.0).all()
    if dst is not None:
        near(dst[0], ref, size, name)
        assert torch.equal(dst[0][torch.from_numpy(live).cuda()], rows[torch.from_numpy(slots[live]).cuda()])


def test_latent_cache_write_of_strided_rows_and_zeros():
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(8)
    wide = rounded(rng, (1, 40, 640), "bf16")
    kv = wide[:, :, 32:608]
    kv[0, 3] = 0  # a padding row
    cache = ab.new_latent_cache(4, 16, torch.bfloat16)
    w = rounded(rng, (512,), "bf16")
    ab.latent_cache_write(kv, i32(np.arange(40)), cache, norm_weight=w, norm_eps=1e-6)
    ref, size = oracle.cache_rows(f64(kv)[0], f64(w), 1e-6)
    near(cache.view(-1, 576)[:40], ref, size, "bf16")
    assert (cache.view(-1, 576)[3] == 0).all() and (cache.view(-1, 576)[40:] == 0).all()
    # a cache of wider rows
    big = torch.zeros(2, 32, 600, dtype=torch.bfloat16, device="cuda")
    ab.latent_cache_write(kv, i32(np.arange(63, 23, -1)), big[:, :, :576], norm_weight=w)
    assert torch.equal(big.view(64, 600)[63 - 39:, :576].flip(0), cache.view(-1, 576)[:40]) and (big[:, :, 576:] == 0).all()
    ab.latent_cache_write(kv[:, :0], i32([]), cache)  # no tokens
