"""More heads a group than a call over lists takes: calls on views."""
import numpy as np
import pytest

from oracle import latent as oracle
from test_gpu_latent import near
from test_gpu_rope import f64, i32, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [5, 130])  # lists in parts, and whole
def test_lists_of_more_heads_by_views(S):
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(S)
    H, G = 192, 2  # 96 heads a group
    q, kv = rounded(rng, (1, S, H, 576), "bf16"), rounded(rng, (1, 200, G, 576), "bf16")
    idx = rng.integers(-1, 200, (1, S, G, 140))
    with pytest.raises(ab.AttnBwdError):
        ab.sparse_forward(q, kv, i32(idx), 0.05)
    o, lse = torch.full((1, S, H, 512), float("nan"), dtype=q.dtype, device="cuda"), torch.full((1, H, S), float("nan"), device="cuda")
    for g in range(G):
        for a, e in ((0, 64), (64, 96)):
            h = slice(g * 96 + a, g * 96 + e)
            ab.sparse_forward(q[:, :, h], kv[:, :, g:g + 1], i32(idx)[:, :, g:g + 1], 0.05, out=(o[:, :, h], lse[:, h]))
    near(o, lse.transpose(1, 2), oracle.list_forward(f64(q), f64(kv), idx, 0.05), "bf16")
