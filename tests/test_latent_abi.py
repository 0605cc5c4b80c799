"""Rotary positions and latent attention without a GPU: what the entry points
export and refuse before anything is queued, the frequency tables, and pins of the
oracle."""
import ctypes
import math
import os
import random
import re

import numpy as np
import pytest

import __graft_entry__
from oracle import attention, latent as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 4096  # an aligned address that no refused call may touch
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ab():
    __graft_entry__.build()
    import attention_backward_gb300 as ab

    return ab


@pytest.mark.parametrize("header,names", [
    ("attn_rope.h", {"attn_rope"}),
    ("attn_latent.h", {"attn_latent_cache_write", "attn_fwd_latent_cache_workspace_size", "attn_fwd_latent_cache",
                       "attn_fwd_sparse", "attn_fwd_sparse_workspace_size", "attn_fwd_latent",
                       "attn_fwd_latent_workspace_size"})])
def test_declared_symbols_are_exported(ab, header, names):
    src = open(os.path.join(ROOT, "include", header)).read()
    assert set(re.findall(r"ATTN_BWD_API\s+[\w\s\*]+?\b(attn_\w+)\s*\(", src)) == names
    for n in names:
        assert hasattr(ab.library(), n), n


def call(ab, fn, args, **kw):
    a = dict(args)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update({k: ab._binding.Strides(*v) if isinstance(v, tuple) else v for k, v in kw.items()})
    return getattr(ab.library(), fn)(*a.values())


# ------------------------------------------------------------------ rotary positions


def tensor(ab, **kw):
    t = dict(x=A, sx=(4096, 1024, 128), y=A * 8, sy=(4096, 1024, 128), H=8, D=128, start=0)
    assert set(kw) <= set(t)
    t.update(kw)
    flat = [x for v in t.values() for x in (v if isinstance(v, tuple) else (v,))]
    return ctypes.byref(ab._latent._RopeTensor(*flat))


def rope_args(ab):
    return dict(q=tensor(ab), k=None, B=2, S=3, dtype=0, pos=A, pos_b=0, steps=A, R=64, scale=1.0, inter=0, inverse=0,
                stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(D=100), INVALID),
    (dict(start=-8), INVALID), (dict(start=4), INVALID), (dict(start=72), INVALID), (dict(D=56), INVALID),
    (dict(x=A + 8), INVALID), (dict(y=A + 2), INVALID), (dict(sx=(4096, 1024, 4)), INVALID),
    (dict(sy=(4096, 0, 128)), INVALID), (dict(sy=(-8, 1024, 128)), INVALID), (dict(D=1032), UNSUPPORTED),
    (dict(H=(1 << 20) + 1), UNSUPPORTED), (dict(H=2 ** 63 - 1), UNSUPPORTED)])
def test_rope_bad_tensors(ab, kw, want):
    assert call(ab, "attn_rope", rope_args(ab), q=tensor(ab, **kw)) == want
    assert call(ab, "attn_rope", rope_args(ab), k=tensor(ab, **kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(B=0), INVALID), (dict(S=-1), INVALID), (dict(pos=None), INVALID),
    (dict(pos=A + 2), INVALID), (dict(steps=None), INVALID), (dict(steps=A + 4), INVALID), (dict(pos_b=-1), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(R=0), INVALID), (dict(R=24), UNSUPPORTED),
    (dict(R=1040), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(S=1 << 31), UNSUPPORTED),
    (dict(S=1 << 28), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED), (dict(S=0, pos=None), OK)])
def test_rope_refusals(ab, kw, want):
    assert call(ab, "attn_rope", rope_args(ab), **kw) == want


def test_frequencies(ab):
    f, one = ab.rope_frequencies(64)
    assert one == 1.0 and f[0] == 1.0 and f == [10000.0 ** (-i / 32) for i in range(32)]
    assert np.allclose(ab.rope_frequencies(64, scaling="linear", factor=4.0)[0], np.array(f) / 4, rtol=1e-15)
    b = ab.rope_frequencies(64, scaling="base", factor=8.0)[0]
    assert b[0] == 1.0 and abs(b[-1] * 8 / f[-1] - 1) < 1e-12  # the slowest pair: all of the factor
    p, scale = ab.rope_frequencies(64, scaling="parts", factor=8.0, original_length=4096)
    turns = np.array(f) * 4096 / (2 * np.pi)
    r = np.array(p) / np.array(f)
    assert (r[turns > 64] == 1).all() and np.allclose(r[turns < 0.5], 1 / 8) and (np.diff(r) <= 1e-15).all()
    assert abs(scale - (1 + math.log(8) / 10)) < 1e-15


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0), dict(base=INF), dict(factor=0.0),
                                dict(factor=NAN), dict(scaling="cubic"), dict(scaling="base", rotary_dim=2),
                                dict(scaling="parts"), dict(scaling="parts", original_length=0),
                                dict(scaling="parts", original_length=100, beta_fast=1.0, beta_slow=2.0)])
def test_frequency_refusals(ab, kw):
    with pytest.raises(ab.AttnBwdError):
        ab.rope_frequencies(**{"rotary_dim": 64, **kw})


def test_table_holds_every_fraction_of_a_turn(ab):
    """64-bit steps: positions up to 2^31 keep their fraction of a turn to 2^-30."""
    table = ab.rope_table(128, base=500000.0, scaling="parts", factor=32.0, original_length=8192, device="cpu")
    f, scale = ab.rope_frequencies(128, base=500000.0, scaling="parts", factor=32.0, original_length=8192)
    assert table.scale == scale and ab.rope_table(128, scale=0.5, device="cpu").scale == 0.5
    from fractions import Fraction

    for s, w in zip(table.steps.tolist(), f):
        exact = Fraction(w / (2 * math.pi))
        for pos in (1, 131071, 2 ** 31 - 1, -5):
            got = Fraction((pos * s) % 2 ** 64, 2 ** 64)
            off = (got - pos * exact) % 1
            assert min(off, 1 - off) < Fraction(1, 2 ** 30)


# ------------------------------------------------------------------ the cache


def rows(ab, **kw):
    c = dict(rows=A, row_stride=576, num_blocks=32, page_size=16)
    assert set(kw) <= set(c)
    c.update(kw)
    return ctypes.byref(ab._latent._Rows(*c.values()))


def write_args(ab):
    return dict(kv=A, kv_stride=576, slots=A, T=3, dtype=0, weight=None, eps=1e-6, pos=None, steps=None, scale=1.0,
                inter=0, cache=rows(ab), out=None, out_stride=0, stream=None)


def attend_args(ab):
    S = ab._binding.Strides
    return dict(q=A, sq=S(1, 4608, 576), T=3, H=8, dtype=0, scale=0.1, cache=rows(ab), table=A, stride=8, width=8, cu=A,
                kv=A, n=2, causal=1, o=A, so=S(1, 4096, 512), lse=A, sl=S(1, 1, 3), ws=A,
                ws_bytes=ab.latent_cache_workspace_size(), stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=None), INVALID), (dict(rows=A + 8), INVALID), (dict(row_stride=572), INVALID), (dict(row_stride=568), INVALID),
    (dict(row_stride=0), INVALID), (dict(num_blocks=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=256), UNSUPPORTED), (dict(num_blocks=1 << 27), UNSUPPORTED)])
def test_bad_caches(ab, kw, want):
    assert call(ab, "attn_latent_cache_write", write_args(ab), cache=rows(ab, **kw)) == want
    assert call(ab, "attn_fwd_latent_cache", attend_args(ab), cache=rows(ab, **kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kv=None), INVALID), (dict(kv=A + 8), INVALID), (dict(kv_stride=575), INVALID), (dict(kv_stride=568), INVALID),
    (dict(slots=None), INVALID), (dict(slots=A + 1), INVALID), (dict(T=-1), INVALID), (dict(cache=None), INVALID),
    (dict(weight=A + 8), INVALID), (dict(weight=A, eps=-1.0), INVALID), (dict(weight=A, eps=NAN), INVALID),
    (dict(weight=A, eps=INF), INVALID), (dict(pos=A), INVALID), (dict(steps=A), INVALID), (dict(pos=A + 2, steps=A), INVALID),
    (dict(pos=A, steps=A + 4), INVALID), (dict(pos=A, steps=A, scale=NAN), INVALID), (dict(out=A * 2), INVALID),
    (dict(out=A * 2, out_stride=568), INVALID), (dict(out=A * 2 + 2, out_stride=576), INVALID),
    (dict(out=A, out_stride=584), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(T=(1 << 31) - 4095), UNSUPPORTED),
    (dict(T=0, kv=None, slots=None), OK)])
def test_cache_write_refusals(ab, kw, want):
    assert call(ab, "attn_latent_cache_write", write_args(ab), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(table=None), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID), (dict(ws=None), INVALID), (dict(cache=None), INVALID),
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(n=0), INVALID), (dict(width=0), INVALID), (dict(stride=7), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(q=A + 8), INVALID),
    (dict(o=A + 2), INVALID), (dict(ws=A + 8), INVALID), (dict(lse=A + 2), INVALID), (dict(kv=A + 2), INVALID),
    (dict(sq=(1, 4608, 4)), INVALID), (dict(so=(1, 0, 512)), INVALID), (dict(sl=(1, 0, 3)), INVALID),
    (dict(dtype=7), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(T=0, H=1 << 31), UNSUPPORTED),
    (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(width=1 << 27, stride=1 << 27), UNSUPPORTED), (dict(ws_bytes=255), WORKSPACE),
    (dict(T=0, q=None, ws=None), OK)])
def test_cache_attention_refusals(ab, kw, want):
    assert call(ab, "attn_fwd_latent_cache", attend_args(ab), **kw) == want


def test_one_byte_less_workspace_is_refused(ab):
    n = ab.latent_cache_workspace_size()
    assert n > 256 and call(ab, "attn_fwd_latent_cache", attend_args(ab), ws_bytes=n - 1) == WORKSPACE


# ------------------------------------------------------------------ lists and the expanded form


def sparse_args(ab):
    S = ab._binding.Strides
    return dict(q=A, sq=S(36864, 9216, 576), kv=A, skv=S(1152 * 9, 1152, 576), idx=A, si=S(100, 20, 10), B=1, S=4, SKV=9,
                H=16, HKV=2, DQK=576, DV=512, topk=10, dtype=0, scale=0.1, o=A, so=S(32768, 8192, 512), lse=A,
                sl=S(64, 1, 4), ws=A, ws_bytes=256, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(kv=None), INVALID), (dict(idx=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(B=0), INVALID), (dict(S=0), INVALID), (dict(SKV=0), INVALID),
    (dict(H=0), INVALID), (dict(H=15), INVALID), (dict(topk=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=NAN), INVALID), (dict(q=A + 8), INVALID), (dict(kv=A + 8), INVALID), (dict(idx=A + 2), INVALID),
    (dict(lse=A + 1), INVALID), (dict(ws=A + 4), INVALID), (dict(sq=(36864, 9216, 4)), INVALID),
    (dict(so=(0, 8192, 512)), INVALID), (dict(si=(-1, 20, 10)), INVALID), (dict(sl=(64, -1, 4)), INVALID),
    (dict(DQK=512), UNSUPPORTED), (dict(DV=576), UNSUPPORTED), (dict(H=130), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED),
    (dict(skv=(1152 * 9, 1160, 576)), UNSUPPORTED), (dict(skv=(1152 * 9 + 8, 1152, 576)), UNSUPPORTED),
    (dict(skv=(1136 * 9, 1136, 568)), UNSUPPORTED), (dict(S=1 << 31), UNSUPPORTED), (dict(topk=1 << 31), UNSUPPORTED),
    (dict(ws_bytes=255), WORKSPACE)])
def test_sparse_refusals(ab, kw, want):
    assert call(ab, "attn_fwd_sparse", sparse_args(ab), **kw) == want


def test_sparse_workspace(ab):
    assert ab.sparse_forward_workspace_size(1, 80, 1) == ab.sparse_forward_workspace_size(2, 3, 4) > 256
    assert ab.sparse_forward_workspace_size(1, 81, 1) == ab.sparse_forward_workspace_size(2, 4096, 1) == 256
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 31, 1, 1), (1, 1 << 31, 1)):
        assert ab.sparse_forward_workspace_size(*bad) == 0


def expanded_args(ab, **mask):
    S = ab._binding.Strides
    m = ab._binding.Mask(*{**dict(causal=1, window=-1, cu=None, n=0, kv_len=0), **mask}.values())
    return dict(q=A, sq=S(6144, 768, 192), kn=A, skn=S(8192, 1024, 256), kr=A, skr=S(512, 64, 64), v=A,
                sv=S(8192, 1024, 256), B=1, S=8, H=4, dtype=0, scale=0.1, mask=ctypes.byref(m), o=A,
                so=S(4096, 512, 128), lse=A, sl=S(32, 1, 8), ws=A, ws_bytes=ab.latent_workspace_size(1, 8, 4), stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(kn=None), INVALID), (dict(kr=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(B=0), INVALID), (dict(S=0), INVALID), (dict(H=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=INF), INVALID), (dict(q=A + 8), INVALID), (dict(kr=A + 2), INVALID),
    (dict(v=A + 8), INVALID), (dict(o=A + 8), INVALID), (dict(lse=A + 2), INVALID), (dict(ws=A + 8), INVALID),
    (dict(sq=(6144, 768, 4)), INVALID), (dict(skn=(8192, 0, 256)), INVALID), (dict(skr=(512, 4, 64)), INVALID),
    (dict(skr=(0, 64, 64)), INVALID), (dict(sv=(8192, 1024, 0)), INVALID), (dict(so=(4096, 512, 2)), INVALID),
    (dict(sl=(32, 1, -1)), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(S=1 << 31), UNSUPPORTED), (dict(H=65536), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(ws_bytes=255), WORKSPACE)])
def test_expanded_refusals(ab, kw, want):
    assert call(ab, "attn_fwd_latent", expanded_args(ab), **kw) == want


def test_expanded_workspace(ab):
    n = ab.latent_workspace_size(1, 8, 4)
    assert n > 256 and call(ab, "attn_fwd_latent", expanded_args(ab), ws_bytes=n - 1) == WORKSPACE
    assert ab.latent_workspace_size(1, 8192, 64) == n and ab.latent_workspace_size(1, 256, 1, 300) == 256
    assert ab.latent_workspace_size(1, 256, 1, 3) == n
    for bad in ((0, 8, 4, 0), (1, 0, 4, 0), (1, 8, 0, 0), (1, 8, 4, -1), (1, 8, 4, (1 << 20) + 1), (1, 1 << 31, 1, 0)):
        assert ab.latent_workspace_size(*bad) == 0


@pytest.mark.parametrize("mask,kw,want", [
    (dict(window=0), {}, INVALID), (dict(window=-2), {}, INVALID), (dict(window=8), {}, UNSUPPORTED),
    (dict(kv_len=-1), {}, INVALID), (dict(cu=A, n=0), {}, INVALID), (dict(cu=A, n=(1 << 20) + 1), {}, INVALID),
    (dict(cu=A + 2, n=1), {}, INVALID), (dict(cu=A, n=1), dict(B=2), INVALID), (dict(cu=A, n=1, kv_len=9), {}, INVALID),
    (dict(kv_len=(1 << 31) - 1), {}, UNSUPPORTED)])
def test_expanded_mask_refusals(ab, mask, kw, want):
    assert call(ab, "attn_fwd_latent", expanded_args(ab, **mask), **kw) == want


def test_binding_refuses_host_tensors(ab):
    import torch

    q, i = torch.zeros(1, 2, 4, 576, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    table = ab.rope_table(64, device="cpu")
    with pytest.raises(ab.AttnBwdError):
        ab.rope(q, i, table)
    with pytest.raises(ab.AttnBwdError):
        ab.latent_cache_write(q[:, :, 0], i, torch.zeros(3, 16, 576, dtype=torch.float16))
    with pytest.raises(ab.AttnBwdError):
        ab.forward_latent_cache(q, torch.zeros(3, 16, 576, dtype=torch.float16), i[None], i, i[:1], 0.1)
    with pytest.raises(ab.AttnBwdError):
        ab.sparse_forward(q, q[:, :, :1], torch.zeros(1, 2, 1, 3, dtype=torch.int32))
    with pytest.raises(ab.AttnBwdError):
        ab.forward_latent(q[..., :192], q[..., :128], q[:, :, 0, :64], q[..., :128], 0.1)
    with pytest.raises(ab.AttnBwdError):
        ab.new_latent_cache(3, 16, torch.float32, device="cpu")
    assert ab.new_latent_cache(3, 16, torch.bfloat16, device="cpu").shape == (3, 16, 576)


# ------------------------------------------------------------------ the oracle


def test_binding_refuses_other_types(ab):
    import torch

    x, table = torch.zeros(1, 2, 3, 576), ab.rope_table(64, device="cpu")
    for f in (lambda: ab.rope(x, None, table), lambda: ab.rope(x, [0, 1], table), lambda: ab.rope(x, x, table, start="0"),
              lambda: ab.rope(x, x, table, start=1.5), lambda: ab.rope(x, x, table, k=3), lambda: ab.rope(x, x, table, start=2 ** 70),
              lambda: ab.latent_cache_write(x, x, None), lambda: ab.latent_cache_write(x, x, x, norm_eps="small"),
              lambda: ab.forward_latent_cache(x, x, x, x, x, None), lambda: ab.forward_latent_cache(x, x, x, x, x, 0.1, workspace=7),
              lambda: ab.sparse_forward(x, x, x, dv_dim=None), lambda: ab.forward_latent(x, x, x, x, "0.1"),
              lambda: ab.forward_latent(x, x, x, x, 0.1, stream="0")):
        with pytest.raises((ab.AttnBwdError, TypeError, AttributeError)):
            f()


def test_oracle_turn_is_a_rotation_and_its_transpose():
    rng = np.random.default_rng(0)
    f = [1.0, 0.3, 0.01, 1e-4]
    for inter in (False, True):
        eye = np.eye(12)
        m = oracle.turn(eye, 2, f, 12345, 1.0, inter)[0]
        back = oracle.turn(eye, 2, f, 12345, 1.0, inter, inverse=True)[0]
        assert np.allclose(m @ back, eye, atol=1e-14) and np.allclose(m.T, back, atol=1e-14)
        x, y = rng.standard_normal((2, 12))
        # scores depend on the distance alone
        s = [oracle.turn(x, 2, f, p, 1.0, inter)[0] @ oracle.turn(y, 2, f, p + 7, 1.0, inter)[0] for p in (0, 900)]
        assert abs(s[0] - s[1]) < 1e-12


def test_oracle_forms_agree():
    """Lists of a whole request, its pages and the top-k oracle give one result; with
    projections folded into q and behind o the absorbed form is the expanded one."""
    rng = np.random.default_rng(1)
    L, m, H, P = 37, 5, 3, 16
    kv = rng.standard_normal((48, 576))
    q = rng.standard_normal((m, H, 576))
    table = np.array([[2, 0, 1]])
    cache = np.zeros((3, P, 576))
    cache[table[0]] = kv.reshape(3, P, 576)
    a = oracle.cache_forward(q, cache, table, [0, m], [L], 0.05)
    idx = np.full((1, m, 1, L), -1)
    for i in range(m):
        idx[0, i, 0, :L - m + i + 1] = np.arange(L - m + i + 1)
    b = oracle.list_forward(q[None], kv[None, :, None], idx, 0.05)
    o, lse = attention.sparse_forward(q[None], kv[None, :, None], idx, 0.05, 512, dtype=np.float64)
    assert np.allclose(a.o, b.o[0], atol=1e-12) and np.allclose(a.lse, b.lse[0], atol=1e-12)
    assert np.allclose(o, b.o, atol=1e-12) and np.allclose(lse[0].T, b.lse[0], atol=1e-12)
    wk, wv = rng.standard_normal((2, H, 512, 128)) * 0.05
    qe = rng.standard_normal((L, H, 192))
    qa = np.concatenate([np.einsum("thd,hcd->thc", qe[..., :128], wk), qe[..., 128:]], -1)
    kn, v = (np.einsum("tc,hcd->thd", kv[:L, :512], w)[None] for w in (wk, wv))
    x = oracle.expanded_forward(qe[None], kn, kv[None, :L, 512:], v, 0.07)
    y = oracle.cache_forward(qa, cache, table, [0, L], [L], 0.07)
    assert np.allclose(x.o[0], np.einsum("thc,hcd->thd", y.o, wv), atol=1e-11) and np.allclose(x.lse[0], y.lse, atol=1e-11)


# ------------------------------------------------------------------ the measured cases


def test_measured_cases_hold_what_they_look_up():
    """Drawn cases: pages of every position, bounds of packed sequences, work of at most the listed ones'."""
    import importlib.util

    spec = importlib.util.spec_from_file_location("more_cases", os.path.join(ROOT, "perf", "more_operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    rng, ops = random.Random(5), set()
    most = {}
    for c in cases.listed():
        for k, v in cases.work(c).items():
            most[c["op"], k] = max(v, most.get((c["op"], k), 0))
    for c in cases.listed() + [cases.draw(rng) for _ in range(150)]:
        ops.add(c["op"])
        w = cases.work(c)
        assert all(w[k] <= most[c["op"], k] for k in w)
        if c["op"] in ("write", "cache"):
            ctx, new, kv = cases._lens(c)
            table, nb = cases._pages(c, 3)
            assert sum(new) > 0
            for r, n in enumerate(kv):
                pages = table[r, :(n + c["page"] - 1) // c["page"]]
                assert (pages >= 0).all() and (pages < nb).all()
            assert len(np.unique(table[table >= 0])) == (table >= 0).sum()
        if c["op"] == "prompt" and c["packed"]:
            cu = cases._bounds(c)
            assert len(cu) == c["packed"] + 1 and cu[0] == 0 and cu[-1] == c["s"] and sorted(cu) == cu
        if c["op"] == "rope":
            assert c["rot"] % 16 == 0 and c["sq"] + c["rot"] <= c["dq"]
    assert len(ops) == 5
