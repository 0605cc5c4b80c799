"""Binding of ``include/attn_rope.h`` and ``include/attn_latent.h``: rotary
positions and latent attention.  Argument marshalling only, as in ``_binding``, by the
functions of ``csrc/torch_latent.cpp``.

One step of a server of latent attention (``new_lens`` new tokens a request; ``kv``
[1, T, 576] their latent rows, ``q`` [1, T, H, 576] absorbed queries)::

    table = rope_table(64)                                       # once
    cache = new_latent_cache(num_blocks, page_size, kv.dtype)    # once
    plan = kv_block_tables(ctx_lens, new_lens, block_table, free_blocks,
                           page_size, num_blocks, max_tokens)
    latent_cache_write(kv, plan.slot_map, cache, norm_weight=w,
                       positions=plan.positions, table=table)
    rope(q, plan.positions, table, start=512, out=(q, None))
    o, lse = forward_latent_cache(q, cache, block_table, plan.cu_seqlens,
                                  plan.kv_lens, sm_scale)

Launches go to ``stream``, by default the current stream of the tensors' device,
whichever device is current; outputs and workspaces made here belong to that
stream.  Autograd does not see these calls: gradients are ``rope`` with ``inverse`` and
``sparse_backward``.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
from typing import NamedTuple, Optional

import torch

from . import _binding
from ._binding import AttnBwdError, Strides, c_f32, c_i32, c_i64, c_sz, c_vp
from ._kv_cache import DT

ROW, LAT = 576, 512  # values of a latent row, and of its latent vector

TORCH_LIB_PATH = os.path.join(os.path.dirname(_binding.LIB_PATH), "libattn_torch.so")


class _RopeTensor(ctypes.Structure):  # attn_rope_tensor_t, its strides spelled out
    _fields_ = [("x", c_vp), ("sx_b", c_i64), ("sx_s", c_i64), ("sx_h", c_i64), ("y", c_vp), ("sy_b", c_i64),
                ("sy_s", c_i64), ("sy_h", c_i64), ("H", c_i64), ("D", c_i64), ("start", c_i64)]


class _Rows(ctypes.Structure):  # attn_latent_cache_t
    _fields_ = [("rows", c_vp), ("row_stride", c_i64), ("num_blocks", c_i64), ("page_size", c_i64)]


_binding._SIGS.update({
    "attn_rope": (c_i32, [ctypes.POINTER(_RopeTensor), ctypes.POINTER(_RopeTensor), c_i64, c_i64, c_i32, c_vp, c_i64,
                          c_vp, c_i64, c_f32, c_i32, c_i32, c_vp]),
    "attn_latent_cache_write": (c_i32, [c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_f32, c_vp, c_vp, c_f32, c_i32,
                                        ctypes.POINTER(_Rows), c_vp, c_i64, c_vp]),
    "attn_fwd_latent_cache_workspace_size": (c_sz, []),
    "attn_fwd_latent_cache": (c_i32, [c_vp, Strides, c_i64, c_i64, c_i32, c_f32, ctypes.POINTER(_Rows), c_vp, c_i64,
                                      c_i64, c_vp, c_vp, c_i64, c_i32, c_vp, Strides, c_vp, Strides, c_vp, c_sz,
                                      c_vp]),
    "attn_fwd_sparse_workspace_size": (c_sz, [c_i64, c_i64, c_i64]),
    "attn_fwd_sparse": (c_i32, [c_vp, Strides, c_vp, Strides, c_vp, Strides, c_i64, c_i64, c_i64, c_i64, c_i64, c_i64,
                                c_i64, c_i64, c_i32, c_f32, c_vp, Strides, c_vp, Strides, c_vp, c_sz, c_vp]),
    "attn_fwd_latent_workspace_size": (c_sz, [c_i64, c_i64, c_i64, c_i64]),
    "attn_fwd_latent": (c_i32, [c_vp, Strides, c_vp, Strides, c_vp, Strides, c_vp, Strides, c_i64, c_i64, c_i64, c_i32,
                                c_f32, ctypes.POINTER(_binding.Mask), c_vp, Strides, c_vp, Strides, c_vp, c_sz, c_vp]),
})


class RopeTable(NamedTuple):
    """Frequencies of rotary positions, as ``rope_table`` makes them.  Frequencies f_i of
    another scaling, in radians a position, go in as steps[i] = round(f_i / (2 pi) * 2^64)
    modulo 2^64, less 2^64 from 2^63 on."""
    steps: torch.Tensor  # int64 [R / 2] on the device: turns a position * 2^64 (as uint64)
    scale: float         # factor of the result


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: Optional[int] = None, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(radians a position of each pair, factor of the result), as Python floats.

    ``scaling`` stretches base^(-2i/R) to contexts ``factor`` times longer:
    ``"linear"`` divides every frequency by it; ``"base"`` raises the base to
    base * factor^(R/(R-2)); ``"parts"`` divides those of pairs that turn fewer than
    ``beta_slow`` times in ``original_length`` positions, leaves those of pairs that turn
    more than ``beta_fast`` times, goes from one to the other by a ramp over i (from the
    first pair on at the earliest, past the last one where that turns often enough), and
    scales the result by 1 + ln(factor) / 10 (by 1 where the factor is below 1)."""
    R = rotary_dim
    if R < 2 or R % 2:
        raise AttnBwdError("rotary_dim must be positive and even")
    if not (base > 1 and math.isfinite(base)) or not (factor > 0 and math.isfinite(factor)):
        raise AttnBwdError("base must be above 1 and factor above 0")
    if scaling not in ("none", "linear", "base", "parts"):
        raise AttnBwdError(f"scaling {scaling!r}: none, linear, base or parts")
    if scaling == "base":
        if R == 2:
            raise AttnBwdError("scaling of the base needs more than one pair")
        return [(base * factor ** (R / (R - 2))) ** (-2 * i / R) for i in range(R // 2)], 1.0
    w = [base ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        w = [x / factor for x in w]
    if scaling != "parts":
        return w, 1.0
    if original_length is None or original_length < 1 or not beta_fast > beta_slow > 0:
        raise AttnBwdError("scaling in parts needs original_length and beta_fast > beta_slow > 0")

    def pair_of(turns):  # the i whose pair turns so often in original_length positions
        return R * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

    # (the ramp may end past the last pair, which then keeps a share of its frequency)
    lo, hi = max(0, math.floor(pair_of(beta_fast))), min(R - 1, math.ceil(pair_of(beta_slow)))
    ramp = [1.0 if i >= hi else max(0.0, (i - lo) / max(hi - lo, 1)) for i in range(R // 2)]
    return [x * (1 - r) + x / factor * r for x, r in zip(w, ramp)], 1 + max(0.0, math.log(factor)) / 10


def rope_table(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_length: Optional[int] = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
               scale: Optional[float] = None, device=None) -> RopeTable:
    """The table of ``rope_frequencies``' values on the device; ``scale``
    replaces the factor of the result.  Made once, it serves any number of calls."""
    w, own = rope_frequencies(rotary_dim, base, scaling, factor, original_length, beta_fast, beta_slow)
    steps = [round(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for x in w]
    t = torch.tensor([s - 2 ** 64 if s >= 2 ** 63 else s for s in steps], dtype=torch.int64)
    return RopeTable(t.to(torch.device("cuda" if device is None else device)), own if scale is None else float(scale))


_ops = None


def _operators():
    """The functions of csrc/torch_latent.cpp (raises if they have not been built)."""
    global _ops
    if _ops is None:
        if not os.path.exists(TORCH_LIB_PATH):
            raise AttnBwdError(f"library missing at {TORCH_LIB_PATH}: build it with attention_backward_gb300.build")
        loader = importlib.machinery.ExtensionFileLoader("libattn_torch", TORCH_LIB_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("libattn_torch", loader))
        loader.exec_module(module)
        _ops = {n: getattr(module, n) for n in ("rope", "latent_cache_write", "forward_latent_cache", "sparse_forward",
                                                "forward_latent")}
    return _ops


def _call(name, first, stream, *args):
    """Function ``name`` on ``stream`` (None: the current one of first's device)."""
    if stream is not None:
        if isinstance(stream, torch.cuda.Stream) and isinstance(first, torch.Tensor) and stream.device != first.device:
            raise AttnBwdError("stream belongs to another device than the tensors")
        stream = _binding._stream(stream)
    try:
        return (_ops or _operators())[name](first, *args, stream)
    except RuntimeError as e:
        if isinstance(e, (AttnBwdError, torch.cuda.OutOfMemoryError)):
            raise
        raise AttnBwdError(str(e).split("\nException raised from", 1)[0]) from None


def _table(table):
    if not isinstance(table, RopeTable):
        raise AttnBwdError("table must be a RopeTable (rope_table)")
    return table


def _pair(out):
    if out is None:
        return None, None
    if len(out) != 2:
        raise AttnBwdError("out must be a pair of tensors")
    return out


def rope(q, positions, table: RopeTable, k=None, interleaved: bool = False, start: int = 0, k_start: int = 0,
         inverse: bool = False, out=None, stream=None):
    """(q, k) with columns [start, start + R) of each head of ``q`` [B,S,H,D]
    (``k_start`` of ``k`` [B,S,Hk,Dk], if given) turned to ``positions`` (int32 [S] or [B,S]; see
    attn_rope); R is the table's.  ``inverse`` turns back: given the gradients of a
    call's results it returns those of its inputs.  ``out`` (q', k') writes into
    tensors of the same shapes; the inputs themselves work in place."""
    steps, scale = _table(table)
    return _call("rope", q, stream, positions, steps, scale, k, interleaved, start, k_start, inverse, *_pair(out))


def new_latent_cache(num_blocks: int, page_size: int, dtype, device=None):
    """A zeroed latent cache [num_blocks, page_size, 576] of fp16 or bf16."""
    if dtype not in DT:
        raise AttnBwdError(f"unsupported dtype {dtype}: fp16 or bf16")
    return torch.zeros(num_blocks, page_size, ROW, dtype=dtype, device="cuda" if device is None else device)


def latent_cache_write(kv, slot_map, cache, norm_weight=None, norm_eps: float = 1e-6, positions=None,
                       table: Optional[RopeTable] = None, interleaved: bool = False, out=None, stream=None) -> None:
    """Writes new tokens' latent rows ``kv`` [1,T,576] into the cache at
    ``slot_map`` int32 [T]: the first 512 columns normalised by their root mean square
    and ``norm_weight`` [512] (None: as they are), the last 64 turned to ``positions``
    int32 [T] by ``table`` (both or neither; see attn_latent_cache_write).  ``out``
    [1,T,576], ``kv`` itself among others, gets the same rows."""
    steps, scale = (None, 1.0) if table is None else _table(table)
    _call("latent_cache_write", kv, stream, slot_map, cache, norm_weight, norm_eps, positions, steps, scale, interleaved,
          out)


def latent_cache_workspace_size() -> int:
    """Workspace bytes of forward_latent_cache."""
    return int(_binding.library().attn_fwd_latent_cache_workspace_size())


def forward_latent_cache(q, cache, block_table, cu_seqlens, kv_lens, sm_scale: float, causal: bool = True,
                         workspace=None, out=None, stream=None):
    """O [1,T,H,512] and the natural-log LSE [1,H,T] of packed absorbed queries
    [1,T,H,576] over their requests' cached latent rows (see attn_fwd_latent_cache):
    request n's rows are cu_seqlens[n] to cu_seqlens[n + 1], its keys the first kv_lens[n]
    positions of its ``block_table`` row.  ``out`` (o, lse) and ``workspace`` (uint8,
    latent_cache_workspace_size bytes; one per stream) may be passed to reuse them."""
    return _call("forward_latent_cache", q, stream, cache, block_table, cu_seqlens, kv_lens, sm_scale, causal, workspace,
                 *_pair(out))


def sparse_forward_workspace_size(B: int, S: int, HKV: int) -> int:
    """Workspace bytes of sparse_forward with room to split the lists of few tokens (256 always serve)."""
    return int(_binding.library().attn_fwd_sparse_workspace_size(B, S, HKV))


def sparse_forward(q, kv, idx, sm_scale: Optional[float] = None, dv_dim: int = LAT, workspace=None, out=None,
                   stream=None):
    """O [B,S,H,512] and the natural-log LSE [B,H,S] of top-k sparse attention
    over shared latent rows, as ``sparse_backward`` takes them (see attn_fwd_sparse):
    q [B,S,H,576], kv [B,SKV,HKV,576], idx int32 [B,S,HKV,topk], at most 64 heads a
    group (more: a call for 64 heads each, on views of q, o and lse).  ``out`` (o, lse) and
    ``workspace`` (uint8, at least 256 bytes; one per stream) may be passed to reuse them."""
    return _call("sparse_forward", q, stream, kv, idx, ROW ** -0.5 if sm_scale is None else sm_scale, dv_dim, workspace,
                 *_pair(out))


def latent_workspace_size(B: int, S: int, H: int, num_seqs: int = 0) -> int:
    """Workspace bytes of forward_latent."""
    return int(_binding.library().attn_fwd_latent_workspace_size(B, S, H, num_seqs))


def forward_latent(q, k_nope, k_rope, v, sm_scale: float, causal: bool = True, cu_seqlens=None, workspace=None,
                   out=None, stream=None):
    """O [B,S,H,128] and the natural-log LSE [B,H,S] of the expanded form (see
    attn_fwd_latent): q [B,S,H,192], k_nope and v [B,Sk,H,128] (views of one projection
    serve), k_rope [B,Sk,64] shared by the heads.  Where Sk differs from S, the last
    query stands at the last key.  ``cu_seqlens`` int32 packs sequences (B = 1, Sk = S).
    ``out`` (o, lse) and ``workspace`` (uint8, latent_workspace_size bytes; one per stream)
    may be passed to reuse them."""
    return _call("forward_latent", q, stream, k_nope, k_rope, v, sm_scale, causal, cu_seqlens, workspace, *_pair(out))
