"""Latent attention whose units last longer than a second, the limit of the waits inside one."""
import math

import numpy as np
import pytest

from oracle import latent as oracle
from test_gpu_rope import f64, i32, rounded

pytestmark = pytest.mark.gpu


def test_lists_of_many_rows():
    """One list of 90 million entries, shared by more tokens than the GPU has
    multiprocessors: a CTA's second unit waits for its first, some two seconds, and no wait
    runs out.  The sum of weights has f32 steps: within (additions a thread) 2^-24 of it."""
    import torch

    import attention_backward_gb300 as ab

    rng = np.random.default_rng(1)
    rows, H, topk, name = 64, 16, 90_000_000, "bf16"
    S = torch.cuda.get_device_properties(0).multi_processor_count + 8
    kv = rounded(rng, (1, rows, 1, 576), name)
    q = rounded(rng, (1, 1, H, 576), name).expand(1, S, H, 576).contiguous()
    idx = (torch.arange(topk, dtype=torch.int32, device="cuda") % rows).expand(1, S, 1, topk)
    assert idx.stride(1) == 0
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    o, lse = ab.sparse_forward(q, kv, idx, 0.05, workspace=ws)
    end.record()
    ab.check_error(ws)
    assert begin.elapsed_time(end) > 2000  # (two units: each longer than the limit)
    r = oracle.list_forward(f64(q[:, :1]), f64(kv), np.arange(rows)[None, None, None], 0.05)
    want = r.lse[0, 0] + math.log(topk / rows)
    assert (np.abs(f64(lse)[0] - want[:, None]) <= 1.1 * topk / 64 * 2.0 ** -24 + r.le[0, 0][:, None] + 2.0 ** -18).all()
    assert o.isfinite().all() and torch.equal(o[:, :1].expand_as(o), o)
