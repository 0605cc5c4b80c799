"""Latent attention with scores far beyond what a power of two holds.

One column carries the scores: powers of two of either sign in q, distinct integers of
at most 8 bits times a power of two in the keys.  The scores are then exact in f32 and so
far apart that a row's softmax is shared by the keys of its largest score: O is their mean, and the LSE the
scaled score within the roundings of its scale, products and sum, 4 of them (2^-22 of it).
Every fourth head has ordinary scores, in whose bound the others have no part."""
import numpy as np
import pytest

from oracle import latent as oracle
from test_gpu_latent import near
from test_gpu_rope import EPS, STEP, f64, i32, rounded

pytestmark = pytest.mark.gpu

# type, powers of two in q, power of two of the keys, scale: scaled scores of up to 10^10 to 10^35
SIZES = [("f16", (15, 13, 15), 8, 16.0), ("bf16", (20, 10, 15), 20, 0.05), ("bf16", (52, 50, 60), 50, 0.05),
         ("bf16", (54, 40, 56), 52, 3.0)]
KEYS = 250


def problem(rng, name, powers, power, heads, width, order):
    """q [1, 3, heads, width], whose last column carries the scores, and the keys' last column."""
    import torch

    q = rounded(rng, (1, 3, heads, width), name)
    for h in range(heads):
        if h % 4:
            q[:, :, h] = 0
            q[:, :, h, -1] = (-1) ** (h // 4 + h % 4) * 2.0 ** powers[h % 4 - 1]
        else:
            q[:, :, h, -1] = 0
    m = {"rising": np.arange(KEYS), "falling": np.arange(KEYS)[::-1], "mixed": rng.permutation(KEYS)}[order] + 1
    return q, torch.from_numpy(m * 2.0 ** power).to(q.dtype).cuda()


def check(o, lse, r, name):
    """o [.., heads, dv], lse [.., heads] against r."""
    heads = np.arange(lse.shape[-1])
    plain, far = heads % 4 == 0, heads % 4 != 0
    # the mean of the t <= 20 rows that share the largest score (weights of 2^7 each, without
    # rounding): the output's rounding, and f32 sums, (t + 3) 2^-24 of the sum of |v| at most
    want = r.o[..., far, :]
    tol = EPS[name] * np.abs(want) + 2.0 ** -19 * r.mag[..., far, :] + STEP[name]
    assert (np.abs(f64(o)[..., far, :] - want) <= tol).all()
    assert np.abs(r.lse[..., far]).min() > 1e7 and np.abs(r.lse).max() > 1e9
    assert (np.abs(f64(lse)[..., far] / r.lse[..., far] - 1) <= 2.0 ** -22).all()
    part = oracle.Result((0,), r.o.shape[-1])
    for key in vars(part):
        setattr(part, key, getattr(r, key)[..., plain, :] if getattr(r, key).ndim > r.lse.ndim else getattr(r, key)[..., plain])
    near(o[..., plain, :], lse[..., plain], part, name)


@pytest.mark.parametrize("name,powers,power,scale", SIZES)
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_lists_of_far_scores(name, powers, power, scale, order):
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(power)
    q, last = problem(rng, name, powers, power, 24, 576, order)
    rows = rounded(rng, (1, KEYS, 1, 576), name, 0.125)
    rows[0, :, 0, -1] = last
    idx = np.sort(rng.integers(0, KEYS, (1, 3, 1, 1500)))
    idx[0, 1, 0, 5:] = -1  # few entries, and none
    idx[0, 2] = -1
    r = oracle.list_forward(f64(q), f64(rows), idx, scale)
    for room in (256, ab.sparse_forward_workspace_size(1, 3, 1)):  # whole, and in parts
        ws = torch.empty(room, dtype=torch.uint8, device="cuda")
        o, lse = ab.sparse_forward(q, rows, i32(idx), scale, workspace=ws)
        ab.check_error(ws)
        assert (o[:, 2] == 0).all() and torch.isneginf(lse[:, :, 2]).all()
        live = oracle.Result((0,), 512)
        for key in vars(live):
            setattr(live, key, getattr(r, key)[:, :2])
        check(o[:, :2], lse.transpose(1, 2)[:, :2], live, name)


@pytest.mark.parametrize("name,powers,power,scale", SIZES)
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_cache_of_far_scores(name, powers, power, scale, order):
    import attention_backward_gb300 as ab

    rng = np.random.default_rng(power + 1)
    q, last = problem(rng, name, powers, power, 40, 576, order)
    cache = rounded(rng, (16, 16, 576), name, 0.125)
    table = rng.permutation(16)
    for j in range(KEYS):
        cache[table[j // 16], j % 16, -1] = last[j]
    r = oracle.cache_forward(f64(q)[0], f64(cache), table[None], [0, 3], [KEYS], scale)
    o, lse = ab.forward_latent_cache(q, cache, i32(table[None]), i32([0, 3]), i32([KEYS]), scale)
    check(o[0], lse[0].t(), r, name)


@pytest.mark.parametrize("name,powers,power,scale", SIZES)
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("S,Sk", [(3, KEYS), (2, 2000)])  # whole, and keys in parts
def test_expanded_of_far_scores(name, powers, power, scale, order, S, Sk):
    import attention_backward_gb300 as ab

    rng = np.random.default_rng(power + 2)
    q, last = problem(rng, name, powers, power, 12, 192, order)
    q = q[:, :S].contiguous()
    up, kr = rounded(rng, (1, Sk, 12, 256), name, 0.125), rounded(rng, (1, Sk, 64), name, 0.125)
    kr[0, :, -1] = last[np.sort(rng.integers(0, KEYS, Sk)) if Sk > KEYS else np.arange(Sk)]
    for causal in (True, False):
        r = oracle.expanded_forward(f64(q), f64(up[..., :128]), f64(kr), f64(up[..., 128:]), scale, causal)
        o, lse = ab.forward_latent(q, up[..., :128], kr, up[..., 128:], scale, causal=causal)
        check(o, lse.transpose(1, 2), r, name)
