"""Binding of ``include/attn_rope.h`` and ``include/attn_latent.h``: rotary
positions and latent attention.  Argument marshalling only, as in ``_binding``.

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
stream.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import _binding
from ._binding import AttnBwdError, Strides, c_f32, c_i32, c_i64, c_sz, c_vp
from ._kv_cache import DT, _device, _on, _run, _strides, _table, _vec

ROW, LAT, ROT = 576, 512, 64  # a latent row, its latent vector, its rotated columns
NOPE, DV = 128, 128           # the expanded form's own key columns and values a head

_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8


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
    "attn_fwd_sparse": (c_i32, [c_vp, Strides, c_vp, Strides, c_vp, Strides, c_i64, c_i64, c_i64, c_i64, c_i64, c_i64,
                                c_i64, c_i64, c_i32, c_f32, c_vp, Strides, c_vp, Strides, c_vp, c_sz, c_vp]),
    "attn_fwd_latent": (c_i32, [c_vp, Strides, c_vp, Strides, c_vp, Strides, c_vp, Strides, c_i64, c_i64, c_i64, c_i32,
                                c_f32, ctypes.POINTER(_binding.Mask), c_vp, Strides, c_vp, Strides, c_vp, c_sz, c_vp]),
})


class RopeTable(NamedTuple):
    """Frequencies of rotary positions, as ``rope_table`` makes them."""
    steps: torch.Tensor  # int64 [R / 2] on the device: turns a position * 2^64 (as uint64)
    scale: float         # factor of the result


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: Optional[int] = None, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(radians a position of each pair, factor of the result), as Python floats.

    ``scaling`` stretches base^(-2i/R) to contexts ``factor`` times longer:
    ``"linear"`` divides every frequency by it; ``"base"`` raises the base to
    base * factor^(R/(R-2)); ``"parts"`` divides those of pairs that turn fewer than
    ``beta_slow`` times in ``original_length`` positions, leaves those of pairs that turn
    more than ``beta_fast`` times, goes from one to the other by a ramp over i, and
    scales the result by 1 + ln(factor) / 10."""
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

    lo, hi = max(0, math.floor(pair_of(beta_fast))), min(R // 2 - 1, math.ceil(pair_of(beta_slow)))
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(R // 2)]
    return [x * (1 - r) + x / factor * r for x, r in zip(w, ramp)], 1 + math.log(factor) / 10


def rope_table(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_length: Optional[int] = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
               scale: Optional[float] = None, device=None) -> RopeTable:
    """The table of ``rope_frequencies``' values on the device; ``scale``
    replaces the factor of the result.  Made once, it serves any number of calls."""
    w, own = rope_frequencies(rotary_dim, base, scaling, factor, original_length, beta_fast, beta_slow)
    steps = [round(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for x in w]
    t = torch.tensor([s - 2 ** 64 if s >= 2 ** 63 else s for s in steps], dtype=torch.int64)
    return RopeTable(t.to(torch.device("cuda" if device is None else device)), own if scale is None else float(scale))


def _dt(name, t):
    dt = DT.get(t.dtype)
    if dt is None:
        raise AttnBwdError(f"{name}: unsupported dtype {t.dtype}: fp16 or bf16")
    return dt


def _steps(table, device, R=None):
    if not isinstance(table, RopeTable):
        raise AttnBwdError("table must be a RopeTable (rope_table)")
    t = table.steps
    if not isinstance(t, torch.Tensor) or t.device != device:
        _on(device, table=t)
    if t.dtype != _I64 or t.dim() != 1 or not t.is_contiguous() or (R is not None and t.shape[0] != R // 2):
        raise AttnBwdError("the table's steps must be a contiguous int64 vector" + ("" if R is None else f" of {R // 2}"))
    return t.data_ptr(), t.shape[0] * 2


def _rope_tensor(name, x, first, y):
    """The C tensor of x turned into y (None: a new one), and y."""
    if y is None:
        y = torch.empty_like(x)
    else:
        _on(x.device, **{name: y})
        if y.dtype != x.dtype:
            raise AttnBwdError(f"{name} must have its input's dtype")
    sx, shape = _strides(name, x), x.shape
    sy = sx if y is x or y.stride() == x.stride() and y.shape == shape else _strides(name, y, shape)
    return _RopeTensor(x.data_ptr(), *sx, y.data_ptr(), *sy, shape[2], shape[3], first), y


def rope(q, positions, table: RopeTable, k=None, interleaved: bool = False, start: int = 0, k_start: int = 0,
         inverse: bool = False, out=None, stream=None):
    """(q, k) with columns [start, start + R) of each head of ``q`` [B,S,H,D]
    (``k_start`` of ``k`` [B,S,Hk,Dk], if given) turned to ``positions`` (int32 [S] or [B,S]; see
    attn_rope); R is the table's.  ``inverse`` turns back: given the gradients of a
    call's results it returns those of its inputs.  ``out`` (q', k') writes into
    tensors of the same shapes; the inputs themselves work in place."""
    device = _device("q", q)
    if not isinstance(positions, torch.Tensor) or positions.device != device:
        _on(device, positions=positions)
    dt = _dt("q", q)
    steps, R = _steps(table, device)
    if q.dim() != 4:
        raise AttnBwdError("q must be a 4-D tensor")
    B, S = q.shape[:2]
    if k is not None:
        _on(device, k=k)
        if k.dtype != q.dtype or k.dim() != 4 or k.shape[:2] != q.shape[:2]:
            raise AttnBwdError("k must have q's dtype, batch and length")
    pos_b = 0
    if positions.dim() == 2:
        pos_b = positions.stride(0) if B > 1 else 0
    if (positions.dtype != _I32 or positions.shape not in ((S,), (B, S)) or (S > 1 and positions.stride(-1) != 1) or
            pos_b < 0):
        raise AttnBwdError(f"positions must be int32 [{S}] or [{B}, {S}] with contiguous rows")
    if out is not None and (len(out) != 2 or out[0] is None or (k is None) != (out[1] is None)):
        raise AttnBwdError("out must be (q, k), k None where none is given")

    def body(ptr):
        tq, yq = _rope_tensor("q", q, start, None if out is None else out[0])
        tk = yk = None
        if k is not None:
            tk, yk = _rope_tensor("k", k, k_start, None if out is None else out[1])
            tk = ctypes.byref(tk)
        _binding._status(_binding.library().attn_rope(
            ctypes.byref(tq), tk, B, S, dt, positions.data_ptr(), pos_b, steps, R, table.scale,
            1 if interleaved else 0, 1 if inverse else 0, ptr), "attn_rope")
        return yq, yk

    return _run(device, stream, body)


def new_latent_cache(num_blocks: int, page_size: int, dtype, device=None):
    """A zeroed latent cache [num_blocks, page_size, 576] of fp16 or bf16."""
    if dtype not in DT:
        raise AttnBwdError(f"unsupported dtype {dtype}: fp16 or bf16")
    return torch.zeros(num_blocks, page_size, ROW, dtype=dtype, device="cuda" if device is None else device)


def _rows(cache):
    if cache.dim() != 3 or cache.shape[2] != ROW or cache.stride(2) != 1:
        raise AttnBwdError(f"cache must be [num_blocks, page_size, {ROW}] with contiguous rows")
    nb, page, _ = cache.shape
    row = cache.stride(1) if page > 1 else cache.stride(0)
    if nb > 1 and page > 1 and cache.stride(0) != page * row:
        raise AttnBwdError("cache must have evenly spaced rows (stride(0) = page_size * stride(1))")
    if nb == 1 and page == 1:
        row = ROW
    return _Rows(cache.data_ptr(), row, nb, page)


def _row_stride(name, t, T):
    if t.shape != (1, T, ROW) or t.stride(2) != 1:
        raise AttnBwdError(f"{name} must be [1, T, {ROW}] with contiguous rows")
    return t.stride(1) if T > 1 else ROW


def latent_cache_write(kv, slot_map, cache, norm_weight=None, norm_eps: float = 1e-6, positions=None,
                       table: Optional[RopeTable] = None, interleaved: bool = False, out=None, stream=None) -> None:
    """Writes new tokens' latent rows ``kv`` [1,T,576] into the cache at
    ``slot_map`` int32 [T]: the first 512 columns normalised by their root mean square
    and ``norm_weight`` [512] (None: as they are), the last 64 turned to ``positions``
    int32 [T] by ``table`` (both or neither; see attn_latent_cache_write).  ``out``
    [1,T,576], ``kv`` itself among others, gets the same rows."""
    device = _device("kv", kv)
    _on(device, slot_map=slot_map, cache=cache)
    dt = _dt("kv", kv)
    if kv.dim() != 3 or cache.dtype != kv.dtype:
        raise AttnBwdError(f"kv must be [1, T, {ROW}] of the cache's dtype")
    T = kv.shape[1]
    sk, rows, slots = _row_stride("kv", kv, T), _rows(cache), _vec("slot_map", slot_map, T)
    weight = pos = steps = None
    if norm_weight is not None:
        _on(device, norm_weight=norm_weight)
        if norm_weight.dtype != kv.dtype or norm_weight.shape != (LAT,) or not norm_weight.is_contiguous():
            raise AttnBwdError(f"norm_weight must be a contiguous vector of {LAT} of kv's dtype")
        weight = norm_weight.data_ptr()
    if (positions is None) != (table is None):
        raise AttnBwdError("positions and table go together")
    if table is not None:
        _on(device, positions=positions)
        pos, steps = _vec("positions", positions, T), _steps(table, device, ROT)[0]
    to = so = None
    if out is not None:
        _on(device, out=out)
        if out.dtype != kv.dtype or out.dim() != 3:
            raise AttnBwdError("out must have kv's dtype and shape")
        to, so = out.data_ptr(), _row_stride("out", out, T)
    _run(device, stream, lambda ptr: _binding._status(_binding.library().attn_latent_cache_write(
        kv.data_ptr(), sk, slots, T, dt, weight, norm_eps, pos, steps, 1.0 if table is None else table.scale,
        1 if interleaved else 0, ctypes.byref(rows), to, so or 0, ptr), "attn_latent_cache_write"))


def latent_cache_workspace_size() -> int:
    """Workspace bytes of forward_latent_cache."""
    return int(_binding.library().attn_fwd_latent_cache_workspace_size())


def _outputs(out, workspace, need, o_shape, dtype, device):
    """o, lse [B, H, S], their strides, and address and bytes of the workspace.  A small
    workspace of the call's own lies behind lse (an allocation is a microsecond or two
    of a short call)."""
    B, S, H, D = o_shape
    lse_shape, own = (B, H, S), workspace is None
    if out is None:
        n = B * H * S
        if own and need <= 4096:
            at = -(-n // 64) * 64
            lse = torch.empty(at + need // 4, dtype=_F32, device=device)
            ws, nbytes = lse.data_ptr() + 4 * at, need
            lse = lse.as_strided(lse_shape, (H * S, S, 1))
            own = False
        else:
            lse = torch.empty(lse_shape, dtype=_F32, device=device)
        o = torch.empty(o_shape, dtype=dtype, device=device)
        so, sl = Strides(S * H * D, H * D, D), Strides(H * S or 1, 1, S or 1)
    else:
        o, lse = out
        _on(device, o=o, lse=lse)
        if o.dtype != dtype or lse.dtype != _F32 or lse.shape != lse_shape:
            raise AttnBwdError(f"out must be o (of q's dtype, {list(o_shape)}) and lse (float32 {list(lse_shape)})")
        lb, lh, ls = lse.stride()
        so = Strides(*_strides("o", o, o_shape))
        sl = Strides(lb if B > 1 else 1, ls if S > 1 else 1, lh if H > 1 else 1)
    keep = None
    if workspace is not None:
        _on(device, workspace=workspace)
        if not workspace.is_contiguous():
            raise AttnBwdError("workspace must be contiguous")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif own:
        keep = torch.empty(need, dtype=_U8, device=device)
        ws, nbytes = keep.data_ptr(), need
    return o, lse, so, sl, ws, nbytes, keep


def forward_latent_cache(q, cache, block_table, cu_seqlens, kv_lens, sm_scale: float, causal: bool = True,
                         workspace=None, out=None, stream=None):
    """O [1,T,H,512] and the natural-log LSE [1,H,T] of packed absorbed queries
    [1,T,H,576] over their requests' cached latent rows (see attn_fwd_latent_cache):
    request n's rows are cu_seqlens[n] to cu_seqlens[n + 1], its keys the first kv_lens[n]
    positions of its ``block_table`` row.  ``out`` (o, lse) and ``workspace`` (uint8,
    latent_cache_workspace_size bytes; one per stream) may be passed to reuse them."""
    device = _device("q", q)
    _on(device, cache=cache, block_table=block_table, cu_seqlens=cu_seqlens, kv_lens=kv_lens)
    dt, rows = _dt("q", q), _rows(cache)
    sq = Strides(*_strides("q", q))
    b, T, H, D = q.shape
    if b != 1 or D != ROW or cache.dtype != q.dtype:
        raise AttnBwdError(f"q must be [1, T, H, {ROW}] of the cache's dtype")
    n = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    lens, cu = _vec("kv_lens", kv_lens, n), _vec("cu_seqlens", cu_seqlens, n + 1)
    table, stride, width = _table(block_table, n)
    lib = _binding.library()

    def body(ptr):
        o, lse, so, sl, ws, nbytes, keep = _outputs(out, workspace, lib.attn_fwd_latent_cache_workspace_size(),
                                                    (1, T, H, LAT), q.dtype, device)
        _binding._status(lib.attn_fwd_latent_cache(
            q.data_ptr(), sq, T, H, dt, sm_scale, ctypes.byref(rows), table, stride, width, cu, lens, n,
            1 if causal else 0, o.data_ptr(), so, lse.data_ptr(), sl, ws, nbytes, ptr), "attn_fwd_latent_cache")
        return o, lse

    return _run(device, stream, body)


def sparse_forward(q, kv, idx, sm_scale: Optional[float] = None, dv_dim: int = LAT, workspace=None, out=None,
                   stream=None):
    """O [B,S,H,512] and the natural-log LSE [B,H,S] of top-k sparse attention
    over shared latent rows, as ``sparse_backward`` takes them (see attn_fwd_sparse):
    q [B,S,H,576], kv [B,SKV,HKV,576], idx int32 [B,S,HKV,topk]."""
    device = _device("q", q)
    _on(device, kv=kv, idx=idx)
    dt = _dt("q", q)
    sq = Strides(*_strides("q", q))
    B, S, H, D = q.shape
    if kv.dim() != 4 or kv.stride(3) != 1 or kv.dtype != q.dtype or kv.shape[0] != B or kv.shape[3] != D:
        raise AttnBwdError(f"kv must be [{B}, SKV, HKV, {D}] of q's dtype with a contiguous last dimension")
    SKV, HKV = kv.shape[1:3]
    if idx.dtype != _I32 or idx.dim() != 4 or idx.shape[:3] != (B, S, HKV) or (idx.shape[3] > 1 and idx.stride(3) != 1):
        raise AttnBwdError(f"idx must be int32 [{B}, {S}, {HKV}, topk] with unit slot stride")
    # (strides of dimensions of size one, which no address uses, follow from the others)
    row = kv.stride(2) if HKV > 1 else kv.stride(1) if SKV > 1 else kv.stride(0) if B > 1 else D
    skv = Strides(kv.stride(0) if B > 1 else SKV * HKV * row, kv.stride(1) if SKV > 1 else HKV * row, row)
    if sm_scale is None:
        sm_scale = D ** -0.5

    def body(ptr):
        o, lse, so, sl, ws, nbytes, _ = _outputs(out, workspace, 256, (B, S, H, dv_dim), q.dtype, device)
        _binding._status(_binding.library().attn_fwd_sparse(
            q.data_ptr(), sq, kv.data_ptr(), skv, idx.data_ptr(), Strides(*idx.stride()[:3]), B, S, SKV, H, HKV, D,
            dv_dim, idx.shape[3], dt, sm_scale, o.data_ptr(), so, lse.data_ptr(), sl, ws, nbytes, ptr), "attn_fwd_sparse")
        return o, lse

    return _run(device, stream, body)


def forward_latent(q, k_nope, k_rope, v, sm_scale: float, causal: bool = True, cu_seqlens=None, workspace=None,
                   out=None, stream=None):
    """O [B,S,H,128] and the natural-log LSE [B,H,S] of the expanded form (see
    attn_fwd_latent): q [B,S,H,192], k_nope and v [B,Sk,H,128] (views of one projection
    serve), k_rope [B,Sk,64] shared by the heads.  Where Sk differs from S, the last
    query stands at the last key.  ``cu_seqlens`` int32 packs sequences (B = 1, Sk = S)."""
    device = _device("q", q)
    _on(device, k_nope=k_nope, k_rope=k_rope, v=v)
    dt = _dt("q", q)
    sq = Strides(*_strides("q", q))
    B, S, H, D = q.shape
    Sk = k_nope.shape[1] if k_nope.dim() == 4 else -1
    if D != NOPE + ROT:
        raise AttnBwdError(f"q must be [B, S, H, {NOPE + ROT}]")
    for name, t in (("k_nope", k_nope), ("k_rope", k_rope), ("v", v)):
        if t.dtype != q.dtype:
            raise AttnBwdError(f"{name} must have q's dtype")
    sk, sv = (Strides(*_strides(n, t, (B, Sk, H, w))) for n, t, w in (("k_nope", k_nope, NOPE), ("v", v, DV)))
    if k_rope.shape != (B, Sk, ROT) or k_rope.stride(2) != 1:
        raise AttnBwdError(f"k_rope must be [{B}, {Sk}, {ROT}] with contiguous rows")
    sr = Strides(k_rope.stride(0) if B > 1 else 128, k_rope.stride(1) if Sk > 1 else 128, 128)
    if cu_seqlens is not None:
        _on(device, cu_seqlens=cu_seqlens)
        _vec("cu_seqlens", cu_seqlens)
    mask = _binding._mask(causal, -1, cu_seqlens, S, Sk)

    def body(ptr):
        o, lse, so, sl, ws, nbytes, _ = _outputs(out, workspace, 256, (B, S, H, DV), q.dtype, device)
        _binding._status(_binding.library().attn_fwd_latent(
            q.data_ptr(), sq, k_nope.data_ptr(), sk, k_rope.data_ptr(), sr, v.data_ptr(), sv, B, S, H, dt, sm_scale,
            ctypes.byref(mask), o.data_ptr(), so, lse.data_ptr(), sl, ws, nbytes, ptr), "attn_fwd_latent")
        return o, lse

    return _run(device, stream, body)
