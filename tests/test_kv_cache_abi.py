"""The paged 8-bit cache entry points without a GPU: what they export, what
they refuse before anything is queued, and pins of their oracle."""
import ctypes
import os
import re

import numpy as np
import pytest

import __graft_entry__
from oracle import attention, kv_cache as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 4096  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def ab():
    __graft_entry__.build()
    import attention_backward_gb300 as ab

    return ab


def test_declared_symbols_are_exported(ab):
    src = open(os.path.join(ROOT, "include", "attn_kv_cache.h")).read()
    names = set(re.findall(r"ATTN_BWD_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", src))
    assert names == {"attn_kv_block_tables", "attn_kv_cache_write", "attn_fwd_kv_cache",
                     "attn_fwd_kv_cache_workspace_size"}
    for n in names:
        assert hasattr(ab.library(), n), n


def call(ab, fn, args, **kw):
    a = dict(args)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return getattr(ab.library(), fn)(*a.values())


TABLES = dict(ctx=A, new=A + 64, n=4, table=A * 2, stride=8, width=8, free=A * 3, num_free=16, start=None, page=16,
              blocks=32, tokens=0, cu=A * 4, kv=A * 5, slots=None, positions=None, counts=A * 6, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(counts=None), INVALID), (dict(n=0), INVALID),
    (dict(stride=7), INVALID), (dict(width=0), INVALID), (dict(num_free=-1), INVALID), (dict(blocks=0), INVALID),
    (dict(tokens=-1), INVALID), (dict(tokens=5), INVALID), (dict(tokens=5, slots=A), INVALID), (dict(page=0), INVALID),
    (dict(ctx=A + 2), INVALID), (dict(start=A + 1), INVALID), (dict(counts=A + 3), INVALID), (dict(kv=A), INVALID),
    (dict(kv=A + 64), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=256), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(blocks=1 << 27), UNSUPPORTED),
    (dict(width=1 << 27, stride=1 << 27), UNSUPPORTED), (dict(num_free=1 << 31), UNSUPPORTED),
    (dict(tokens=1 << 31, slots=A, positions=A), UNSUPPORTED)])
def test_block_tables_refusals(ab, kw, want):
    assert call(ab, "attn_kv_block_tables", TABLES, **kw) == want


def cache(ab, **kw):
    c = dict(k=A, sk=(4096, 256, 128), v=A * 8, sv=(4096, 256, 128), k_scale=A * 16, v_scale=A * 17, num_blocks=32,
             page_size=16, HKV=2, D=128)
    assert set(kw) <= set(c)
    c.update(kw)
    flat = [x for v in c.values() for x in (v if isinstance(v, tuple) else (v,))]
    return ctypes.byref(ab._kv_cache._Cache(*flat))


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(k=A + 8), INVALID), (dict(v=A + 1), INVALID), (dict(k_scale=A + 2), INVALID), (dict(num_blocks=0), INVALID),
    (dict(HKV=0), INVALID), (dict(D=0), INVALID), (dict(page_size=0), INVALID), (dict(sk=(4096, 256, 8)), INVALID),
    (dict(sv=(0, 256, 128)), INVALID), (dict(sv=(4096, -256, 128)), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(num_blocks=1 << 27), UNSUPPORTED),
    (dict(HKV=20000), UNSUPPORTED), (dict(num_blocks=1 << 20, HKV=1 << 11), UNSUPPORTED)]


def write_args(ab):
    S = ab._binding.Strides
    return dict(k=A, sk=S(1, 256, 128), v=A, sv=S(1, 256, 128), slots=A, T=3, dtype=0, cache=cache(ab), stream=None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(ab, kw, want):
    assert call(ab, "attn_kv_cache_write", write_args(ab), cache=cache(ab, **kw)) == want
    assert call(ab, "attn_fwd_kv_cache", attend_args(ab), cache=cache(ab, **kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(T=-1), INVALID),
    (dict(k=A + 8), INVALID), (dict(slots=A + 2), INVALID), (dict(sk=(1, 4, 128)), INVALID),
    (dict(sv=(1, 256, 0)), INVALID), (dict(cache=None), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=0, k=None, slots=None), OK)])
def test_cache_write_refusals(ab, kw, want):
    kw = {k: ab._binding.Strides(*v) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert call(ab, "attn_kv_cache_write", write_args(ab), **kw) == want


def attend_args(ab):
    S = ab._binding.Strides
    n = ab.kv_cache_workspace_size(3, 8, 2, 128)
    return dict(q=A, sq=S(1, 1024, 128), T=3, HQ=8, dtype=0, scale=0.1, cache=cache(ab), table=A, stride=8, width=8,
                cu=A, kv=A, n=2, causal=1, window=-1, o=A, so=S(1, 1024, 128), lse=A, sl=S(1, 1, 3), ws=A, ws_bytes=n,
                stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(table=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(ws=None), INVALID), (dict(cache=None), INVALID),
    (dict(T=-1), INVALID), (dict(HQ=0), INVALID), (dict(HQ=7), INVALID), (dict(n=0), INVALID), (dict(width=0), INVALID),
    (dict(stride=7), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(window=0), INVALID),
    (dict(window=-2), INVALID), (dict(q=A + 8), INVALID), (dict(o=A + 2), INVALID), (dict(ws=A + 8), INVALID),
    (dict(lse=A + 2), INVALID), (dict(sq=(1, 1024, 4)), INVALID), (dict(so=(1, 0, 128)), INVALID),
    (dict(sl=(1, 0, 3)), INVALID), (dict(dtype=7), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED),
    (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(width=1 << 27, stride=1 << 27), UNSUPPORTED),
    (dict(ws_bytes=255), WORKSPACE), (dict(T=0, q=None, ws=None), OK)])
def test_attend_refusals(ab, kw, want):
    kw = {k: ab._binding.Strides(*v) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert call(ab, "attn_fwd_kv_cache", attend_args(ab), **kw) == want


def test_one_byte_less_workspace_is_refused(ab):
    n = ab.kv_cache_workspace_size(3, 8, 2, 128)
    assert n > 256 and call(ab, "attn_fwd_kv_cache", attend_args(ab), ws_bytes=n - 1) == WORKSPACE
    for bad in ((-1, 8, 2, 128), (3, 0, 2, 128), (3, 8, 3, 128), (3, 8, 2, 96), (1 << 29, 8, 2, 128)):
        assert ab.kv_cache_workspace_size(*bad) == 0


def test_counts_just_below_two_to_the_31_are_refused(ab):
    """Counts that 32 bits hold, but not with a tile more: refused before anything is read."""
    big = (1 << 31) - 4095
    assert call(ab, "attn_kv_cache_write", write_args(ab), T=big) == UNSUPPORTED
    assert call(ab, "attn_kv_cache_write", write_args(ab), T=(1 << 31) - 1) == UNSUPPORTED
    assert call(ab, "attn_fwd_kv_cache", attend_args(ab), T=big // 8 + 1) == UNSUPPORTED
    assert call(ab, "attn_fwd_kv_cache", attend_args(ab), width=(1 << 27) - 1, stride=1 << 27) == UNSUPPORTED
    assert ab.kv_cache_workspace_size(big, 1, 1, 128) == 0
    assert ab.kv_cache_workspace_size(big - 1, 1, 1, 128) > 0


def test_binding_refuses_host_tensors(ab):
    import torch

    q = torch.zeros(1, 2, 4, 64, dtype=torch.float16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, i = torch.zeros(3, 2), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ab.AttnBwdError):
        ab.forward_kv_cache(q, c, c, s, s, i[None], i, i[:1])
    with pytest.raises(ab.AttnBwdError):
        ab.kv_cache_write(q[:, :, :2], q[:, :, :2], i, c, c, s, s)
    with pytest.raises(ab.AttnBwdError):
        ab.kv_block_tables(i, i, i.expand(2, 2), i, 16, 3, 4)


# ------------------------------------------------------------------ the oracle


def test_oracle_e4m3_matches_torch():
    import torch

    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(every, oracle.E4M3, equal_nan=True)
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * np.exp2(rng.integers(-13, 10, 20000))).astype(np.float32)
    x[:254] = np.delete(every, [127, 255])  # the values themselves, then the middles between them
    x[254:380] = (oracle.E4M3[:126] + oracle.E4M3[1:127]) / 2
    t = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.to_e4m3(x), t)


def test_oracle_attention_is_the_dense_forward():
    """On one request with contiguous pages: the dense oracle on the values."""
    rng = np.random.default_rng(1)
    L, m, HQ, HKV, D, P = 70, 5, 4, 2, 64, 16
    nb = -(-L // P)
    kc, vc = (oracle.to_e4m3(rng.standard_normal((nb, P, HKV, D)) * 50) for _ in range(2))
    ks, vs = (np.exp2(rng.integers(-7, -4, (nb, HKV))) for _ in range(2))
    q = rng.standard_normal((m, HQ, D))
    val = [(oracle.E4M3[c] * s[:, None, :, None]).reshape(nb * P, HKV, D)[None, :L] for c, s in ((kc, ks), (vc, vs))]
    for causal, window in ((False, -1), (True, -1), (True, 9)):
        o, lse = oracle.forward(q, kc, vc, ks, vs, np.arange(nb)[None], [0, m], [L], 0.1, causal, window)[:2]
        ro, rl = attention.forward(q[None], *val, 0.1, causal, window, dtype=np.float64)
        assert np.allclose(o, ro[0], rtol=1e-12, atol=1e-12) and np.allclose(lse, rl[0], rtol=1e-12)


def test_oracle_write_rounds_to_nearest():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((40, 2, 64)) * 10
    cache, scale = oracle.write(x, 16 + np.arange(40), np.zeros((4, 16, 2, 64), np.uint8), np.zeros((4, 2)))
    y = (oracle.E4M3[cache] * scale[:, None, :, None])[1:].reshape(48, 2, 64)[:40]
    s = np.repeat(scale[1:], 16, 0)[:40][:, :, None]
    assert (np.abs(y - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * s).all()
    amax = np.abs(x[:16]).max(axis=(0, 2))
    assert (amax <= 448 * scale[1]).all() and (amax > 224 * scale[1]).all()
