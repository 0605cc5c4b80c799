"""The expanded form over packed batches of very many sequences."""
import numpy as np
import pytest

from oracle import latent as oracle
from test_gpu_latent import near
from test_gpu_rope import EPS, f64, i32, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,longest,H,causal,name", [
    (3000, 5, 3, True, "bf16"), (77, 600, 2, True, "f16"), (700, 40, 1, False, "bf16"), (33, 300, 5, False, "f16")])
def test_many_sequences(n, longest, H, causal, name):
    """Lengths from none to a few tiles; runs of empty sequences at the ends and between."""
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(n)
    lens = rng.integers(0, longest + 1, n)
    lens[:40 if n > 100 else 2] = lens[n // 2:n // 2 + 35] = lens[-3:] = 0
    cu = np.concatenate([[0], np.cumsum(lens)])
    S = int(cu[-1]) + 9
    q, up, kr = rounded(rng, (1, S, H, 192), name), rounded(rng, (1, S, H, 256), name), rounded(rng, (1, S, 64), name)
    ref = oracle.expanded_forward(f64(q), f64(up[..., :128]), f64(kr), f64(up[..., 128:]), 192 ** -0.5, causal, cu)
    ws = torch.full((ab.latent_workspace_size(1, S, H, n),), 255, dtype=torch.uint8, device="cuda")
    out = (torch.full((1, S, H, 128), float("nan"), dtype=q.dtype, device="cuda"), torch.full((1, H, S), float("nan"), device="cuda"))
    o, lse = ab.forward_latent(q, up[..., :128], kr, up[..., 128:], 192 ** -0.5, causal=causal, cu_seqlens=i32(cu), workspace=ws, out=out)
    ab.check_error(ws)
    near(o, lse.transpose(1, 2), ref, name)
    assert o[:, cu[-1]:].isnan().all() and lse[:, :, cu[-1]:].isnan().all()


def test_as_many_sequences_as_a_call_takes():
    """2^20 sequences of up to two tokens: a row that sees one key has that key's value, one
    that sees two their mean by two weights; and the time does not grow with the square of
    the sequences (some 30 ms; two seconds are allowed)."""
    import torch

    import attention_backward_gb300 as ab

    n, name, scale = 1 << 20, "bf16", 192 ** -0.5
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 3, n)
    cu = np.concatenate([[0], np.cumsum(lens)])
    S = int(cu[-1])
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, up, kr = (torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16) for s in ((1, S, 1, 192), (1, S, 1, 256), (1, S, 64)))
    offsets = i32(cu)
    ws = torch.empty(ab.latent_workspace_size(1, S, 1, n), dtype=torch.uint8, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    o, lse = ab.forward_latent(q, up[..., :128], kr, up[..., 128:], scale, cu_seqlens=offsets, workspace=ws)
    end.record()
    ab.check_error(ws)
    assert begin.elapsed_time(end) < 2000
    k, v = torch.cat([up[0, :, 0, :128], kr[0]], 1), up[0, :, 0, 128:]
    first = torch.from_numpy(cu[:-1][lens > 0]).cuda()
    assert torch.equal(o[0, first, 0], v[first])
    second = torch.from_numpy(cu[:-1][lens == 2] + 1).cuda()
    x, a, b = (t.double() for t in (q[0, second, 0], k[second - 1], k[second]))
    s = torch.stack([(x * a).sum(1), (x * b).sum(1)], 1) * scale
    e = 192 * 2.0 ** -23 * scale * (x.abs() * torch.maximum(a.abs(), b.abs())).sum(1) + 2.0 ** -21
    p, va, vb = s.softmax(1), v[second - 1].double(), v[second].double()
    want, mag = p[:, :1] * va + p[:, 1:] * vb, p[:, :1] * va.abs() + p[:, 1:] * vb.abs()
    # roundings of the output and of the weights, errors of the exponents, f32 sums
    tol = EPS[name] * (want.abs() + mag) + (2 * e[:, None] + 2.0 ** -22) * mag + 2.0 ** -25
    assert ((o[0, second, 0].double() - want).abs() <= tol).all()
    assert ((lse[0, 0, second].double() - s.logsumexp(1)).abs() <= e + 2.0 ** -19).all()
