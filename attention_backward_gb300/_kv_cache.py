"""Binding of ``include/attn_kv_cache.h``: serving from a paged 8-bit
key/value cache.  Argument marshalling only, as in ``_binding``.

One step of a server, every tensor on the GPU (``new_lens`` new tokens a
request, their queries, keys and values packed request by request)::

    plan = kv_block_tables(ctx_lens, new_lens, block_table, free_blocks,
                           page_size, num_blocks, max_tokens)
    kv_cache_write(k, v, plan.slot_map, k_cache, v_cache, k_scale, v_scale)
    o, lse = forward_kv_cache(q, k_cache, v_cache, k_scale, v_scale,
                              block_table, plan.cu_seqlens, plan.kv_lens)

The caches are ``torch.float8_e4m3fn`` [num_blocks, page_size, HKV, D] (any
storage order with a contiguous last dimension; ``new_kv_cache`` makes them),
their scales float32 [num_blocks, HKV].  Launches go to ``stream``, by default
the current stream of the tensors' device, whichever device is current; outputs
and workspaces made here belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _binding
from ._binding import AttnBwdError, Strides, c_f32, c_i32, c_i64, c_sz, c_vp

DT = {torch.float16: _binding.DT_F16, torch.bfloat16: _binding.DT_BF16}


_F8, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32


class _Cache(ctypes.Structure):  # attn_kv_cache_t, its strides spelled out
    _fields_ = [("k", c_vp), ("k_b", c_i64), ("k_s", c_i64), ("k_h", c_i64), ("v", c_vp), ("v_b", c_i64),
                ("v_s", c_i64), ("v_h", c_i64), ("k_scale", c_vp), ("v_scale", c_vp), ("num_blocks", c_i64),
                ("page_size", c_i64), ("HKV", c_i64), ("D", c_i64)]


_binding._SIGS.update({
    "attn_kv_block_tables": (c_i32, [c_vp, c_vp, c_i64, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_i64, c_i64, c_i64,
                                     c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "attn_kv_cache_write": (c_i32, [c_vp, Strides, c_vp, Strides, c_vp, c_i64, c_i32, ctypes.POINTER(_Cache), c_vp]),
    "attn_fwd_kv_cache_workspace_size": (c_sz, [c_i64, c_i64, c_i64, c_i64]),
    "attn_fwd_kv_cache": (c_i32, [c_vp, Strides, c_i64, c_i64, c_i32, c_f32, ctypes.POINTER(_Cache), c_vp, c_i64,
                                  c_i64, c_vp, c_vp, c_i64, c_i32, c_i32, c_vp, Strides, c_vp, Strides, c_vp, c_sz,
                                  c_vp]),
})


class KvPlan(NamedTuple):
    """What attn_kv_block_tables makes of a step's request lengths."""
    cu_seqlens: torch.Tensor  # int32 [N + 1]: packed rows of each request
    kv_lens: torch.Tensor     # int32 [N]: tokens of each request with its new ones
    slot_map: torch.Tensor    # int32 [max_tokens]: slot of each new token, -1 behind the last
    positions: torch.Tensor   # int32 [max_tokens]: its position in its request
    counts: torch.Tensor      # int32 [3]: new tokens, pages taken, what did not fit


class _Launch:
    """Context of a call with a stream or device of its own: the tensors' device
    current, work on ``stream`` (None: that device's current stream), new tensors
    made on it."""

    __slots__ = ("device", "stream", "_ctx")

    def __init__(self, device, stream):
        self.device, self.stream, self._ctx = device, stream, None

    def __enter__(self):
        device, stream = self.device, self.stream
        with contextlib.ExitStack() as ctx:
            ctx.enter_context(torch.cuda.device(device))
            if stream is None:
                stream = torch.cuda.current_stream(device)
            elif not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(_binding._stream(stream), device=device)
            if stream.device != device:
                raise AttnBwdError("stream belongs to another device than the tensors")
            ctx.enter_context(torch.cuda.stream(stream))
            self._ctx = ctx.pop_all()
        return stream.cuda_stream

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)


def _run(device, stream, body):
    """body(stream pointer) with ``device`` current.  (The common case, the
    current stream of the current device, takes no context manager: a decode
    step's calls are bound by the host.)"""
    if stream is None and device.index == torch.cuda.current_device():
        return body(_raw_stream(device.index))
    with _Launch(device, stream) as ptr:
        return body(ptr)


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _raw_stream = torch._C._cuda_getCurrentRawStream  # noqa: F811  (the same without a Stream object)


def _on(device, **tensors):
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor) or t.device != device:
            raise AttnBwdError(f"{name} must be a CUDA tensor on the device of the other tensors")


def _device(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise AttnBwdError(f"{name} must be a CUDA tensor")
    return t.device


def _vec(name, t, n=None):
    if t.dtype != _I32 or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise AttnBwdError(f"{name} must be a contiguous int32 vector" + ("" if n is None else f" of {n}"))
    return t.data_ptr()


def _table(t, n):
    if t.dtype != _I32 or t.dim() != 2 or t.shape[0] != n or t.stride(1) != 1:
        raise AttnBwdError(f"block_table must be int32 [{n}, max_blocks] with contiguous rows")
    # (the stride of a single row says nothing)
    return t.data_ptr(), t.stride(0) if n > 1 else max(t.stride(0), t.shape[1]), t.shape[1]


def _strides(name, t, shape=None):
    """Strides of a 4-D tensor; those of dimensions of size one, which no
    address uses, are replaced by a value that passes the checks."""
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise AttnBwdError(f"{name} must be a 4-D tensor" + ("" if shape is None else f" of shape {list(shape)}"))
    b, s, h, d = t.stride()
    if d != 1:
        raise AttnBwdError(f"{name} must have a contiguous head dimension")
    nb, ns, nh, _ = t.shape
    return b if nb > 1 else 128, s if ns > 1 else 128, h if nh > 1 else 128


def _cache(k_cache, v_cache, k_scale, v_scale, device):
    _on(device, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
    if k_cache.dtype != _F8 or v_cache.dtype != _F8:
        raise AttnBwdError("k_cache and v_cache must be float8_e4m3fn")
    sk = _strides("k_cache", k_cache)
    shape = k_cache.shape
    sv = _strides("v_cache", v_cache, shape)
    nb, page, hkv, d = shape
    for t in (k_scale, v_scale):
        if t.dtype != _F32 or t.shape != (nb, hkv) or not t.is_contiguous():
            raise AttnBwdError("k_scale and v_scale must be contiguous float32 [num_blocks, HKV]")
    return _Cache(k_cache.data_ptr(), *sk, v_cache.data_ptr(), *sv, k_scale.data_ptr(), v_scale.data_ptr(), nb, page,
                  hkv, d)


def new_kv_cache(num_blocks: int, page_size: int, HKV: int, D: int, device=None):
    """(k_cache, v_cache, k_scale, v_scale), zeroed.  The pages are stored head
    by head ([num_blocks, HKV, page_size, D] in memory, seen as [num_blocks,
    page_size, HKV, D]), so that what attention reads of a page for one head is
    contiguous."""
    device = torch.device("cuda" if device is None else device)
    kv = [torch.zeros(num_blocks, HKV, page_size, D, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
          .transpose(1, 2) for _ in range(2)]
    return (*kv, *(torch.zeros(num_blocks, HKV, dtype=torch.float32, device=device) for _ in range(2)))


def kv_block_tables(ctx_lens, new_lens, block_table, free_blocks, page_size: int, num_blocks: int, max_tokens: int,
                    free_start=None, out: Optional[KvPlan] = None, stream=None) -> KvPlan:
    """Pages, slots, positions and row ranges of a step's new tokens (see
    attn_kv_block_tables).  ``block_table`` int32 [N, max_blocks] gets the new
    pages' entries in place; ``free_blocks`` int32 holds the free pages from
    entry ``free_start`` (int32 [1] on the device; None: 0) on.  ``out`` reuses
    a plan's tensors (a captured step)."""
    device = _device("ctx_lens", ctx_lens)
    _on(device, new_lens=new_lens, block_table=block_table, free_blocks=free_blocks)
    n = ctx_lens.shape[0] if ctx_lens.dim() == 1 else -1
    ctx, add = _vec("ctx_lens", ctx_lens, n), _vec("new_lens", new_lens, n)
    table, stride, width = _table(block_table, n)
    free = _vec("free_blocks", free_blocks)
    start = None
    if free_start is not None:
        _on(device, free_start=free_start)
        start = _vec("free_start", free_start, 1)
    sizes = (n + 1, n, max_tokens, max_tokens, 3)

    def body(ptr):
        plan, ptrs = out, None
        if plan is None:
            if max_tokens < 0:
                raise AttnBwdError("max_tokens must not be negative")
            buf = torch.empty(sum(sizes), dtype=_I32, device=device)  # one buffer for the five outputs
            plan = KvPlan(*torch.unsafe_split_with_sizes(buf, sizes))  # (split()'s views would cost twice that)
            at, ptrs = buf.data_ptr(), []
            for k in sizes:
                ptrs.append(at)
                at += 4 * k
        else:
            _on(device, **plan._asdict())
            ptrs = [_vec(name, t, k) for name, t, k in zip(plan._fields, plan, sizes)]
        _binding._status(_binding.library().attn_kv_block_tables(
            ctx, add, n, table, stride, width, free, free_blocks.shape[0], start, page_size, num_blocks, max_tokens,
            *ptrs, ptr), "attn_kv_block_tables")
        return plan

    return _run(device, stream, body)


def kv_cache_write(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """Writes new tokens' keys and values, [1,T,HKV,D] fp16 or bf16, into the
    cache at ``slot_map`` int32 [T], rounding to e4m3 with a scale per page and
    KV head (see attn_kv_cache_write)."""
    device = _device("k", k)
    _on(device, v=v, slot_map=slot_map)
    c = _cache(k_cache, v_cache, k_scale, v_scale, device)
    sk = Strides(*_strides("k", k))
    T = k.shape[1]
    shape = (1, T, c.HKV, c.D)
    if k.shape != shape:
        raise AttnBwdError(f"k must be [1, T, {c.HKV}, {c.D}]")
    sv = Strides(*_strides("v", v, shape))
    dt = DT.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise AttnBwdError(f"unsupported dtypes {k.dtype}, {v.dtype}: both fp16 or both bf16")
    slots = _vec("slot_map", slot_map, T)
    _run(device, stream, lambda ptr: _binding._status(_binding.library().attn_kv_cache_write(
        k.data_ptr(), sk, v.data_ptr(), sv, slots, T, dt, ctypes.byref(c), ptr), "attn_kv_cache_write"))


def kv_cache_workspace_size(T: int, HQ: int, HKV: int, D: int) -> int:
    """Workspace bytes of forward_kv_cache for T queries."""
    return int(_binding.library().attn_fwd_kv_cache_workspace_size(T, HQ, HKV, D))


def forward_kv_cache(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, kv_lens,
                     sm_scale: Optional[float] = None, causal: bool = True, window: int = -1, workspace=None, out=None,
                     stream=None):
    """O [1,T,HQ,D] and the natural-log LSE [1,HQ,T] of packed queries
    [1,T,HQ,D] over the cached keys of their requests (see attn_fwd_kv_cache):
    request n's rows are cu_seqlens[n] to cu_seqlens[n + 1], its keys the first
    kv_lens[n] positions of its ``block_table`` row.  ``out`` (o, lse) and
    ``workspace`` (uint8, kv_cache_workspace_size bytes; one per stream) may be
    passed to reuse them."""
    device = _device("q", q)
    _on(device, block_table=block_table, cu_seqlens=cu_seqlens, kv_lens=kv_lens)
    c = _cache(k_cache, v_cache, k_scale, v_scale, device)
    sq = Strides(*_strides("q", q))
    b, T, HQ, D = q.shape
    dt = DT.get(q.dtype)
    if dt is None:
        raise AttnBwdError(f"unsupported dtype {q.dtype}: fp16 or bf16")
    if b != 1 or D != c.D:
        raise AttnBwdError(f"q must be [1, T, HQ, {c.D}]")
    n = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    lens, cu = _vec("kv_lens", kv_lens, n), _vec("cu_seqlens", cu_seqlens, n + 1)
    table, stride, width = _table(block_table, n)
    if sm_scale is None:
        sm_scale = D ** -0.5
    lib = _binding.library()

    def body(ptr):
        if out is None:
            o = torch.empty_like(q, memory_format=torch.contiguous_format)
            lse = torch.empty((1, HQ, T), dtype=_F32, device=device)
            so, sl = Strides(T * HQ * D, HQ * D, D), Strides(1, 1, max(T, 1))
        else:
            o, lse = out
            _on(device, o=o, lse=lse)
            if o.dtype != q.dtype or lse.dtype != _F32 or lse.shape != (1, HQ, T):
                raise AttnBwdError("out must be o (of q's dtype and shape) and lse (float32 [1, HQ, T])")
            so = Strides(*_strides("o", o, q.shape))
            sl = Strides(1, lse.stride(2) if T > 1 else 1, lse.stride(1) if HQ > 1 else 1)
        if workspace is None:
            ws = torch.empty(lib.attn_fwd_kv_cache_workspace_size(T, HQ, c.HKV, D), dtype=torch.uint8, device=device)
            nbytes = ws.numel()
        else:
            ws = workspace
            _on(device, workspace=ws)
            if not ws.is_contiguous():
                raise AttnBwdError("workspace must be contiguous")
            nbytes = ws.numel() * ws.element_size()
        _binding._status(lib.attn_fwd_kv_cache(
            q.data_ptr(), sq, T, HQ, dt, sm_scale, ctypes.byref(c), table, stride, width, cu, lens, n,
            1 if causal else 0, window, o.data_ptr(), so, lse.data_ptr(), sl, ws.data_ptr(), nbytes, ptr),
            "attn_fwd_kv_cache")
        return o, lse

    return _run(device, stream, body)
