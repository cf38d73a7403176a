"""Packed, paged serving operators of libkvc (include/kvc.h): the rotary append
into a block pool and read-only attention over it, pools in the inputs' type or
in 8 bits.

Both take T packed tokens of B sequences: ``cu_seqlens_q`` [B + 1] the packing
offsets (S_b rows each), ``seqlens_k`` [B] the cached positions K_b with the new
ones included, ``block_table`` [B, max_blocks] the pool block of each run of
block_size slots. Argument marshalling only, as in kvc.py: no CPU path.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from .kvc import DTYPES, KvcError, default_scale, library, status_string

#: pool types in 8 bits, kept with one fp32 scale for each (block, head)
EIGHT_BIT = {torch.float8_e4m3fn: 3, torch.float8_e5m2: 4}
_INTEGERS = (torch.int8, torch.uint8, torch.int16, torch.int32, torch.int64)
_POOL_DTYPES = {**DTYPES, **EIGHT_BIT}


class PagedDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("B", "total_q", "max_q", "Hq", "Hk", "D", "Dv", "num_blocks", "block_size",
                 "max_blocks")] + [("dtype", ctypes.c_int32), ("pool_dtype", ctypes.c_int32)]


_lib = None


def _paged_library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = library()
        vp, i64, i32, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
        dp, sp = ctypes.POINTER(PagedDims), ctypes.POINTER(ctypes.c_int64)
        lib.kvc_append_rotary_paged.restype = ctypes.c_int
        lib.kvc_append_rotary_paged.argtypes = [dp, i64, i64, i32, sp] + [vp] * 15
        lib.kvc_attend_paged_path.restype = ctypes.c_char_p
        lib.kvc_attend_paged_path.argtypes = [dp]
        lib.kvc_attend_paged_workspace_bytes.restype = ctypes.c_size_t
        lib.kvc_attend_paged_workspace_bytes.argtypes = [dp]
        lib.kvc_attend_paged.restype = ctypes.c_int
        lib.kvc_attend_paged.argtypes = ([dp, sp] + [vp] * 8 + [f64, f64, vp, i64, vp, vp,
                                                               ctypes.c_size_t, vp, vp])
        _lib = lib
    return _lib


def make_paged_dims(B, total_q, max_q, Hq, Hk, D, Dv, num_blocks, block_size, max_blocks, dtype,
                    pool_dtype=None) -> PagedDims:
    """Sizes of one call; dtype and pool_dtype (default: the dtype) as torch
    dtypes or kvc_dtype codes."""
    code = _POOL_DTYPES.get(dtype, dtype)
    pool = code if pool_dtype is None else _POOL_DTYPES.get(pool_dtype, pool_dtype)
    return PagedDims(B, total_q, max_q, Hq, Hk, D, Dv, num_blocks, block_size, max_blocks, code,
                     pool)


def attend_paged_path(dims: PagedDims) -> str:
    """Name of the kernel attention_over_paged_cache takes for these sizes."""
    name = _paged_library().kvc_attend_paged_path(ctypes.byref(dims))
    if name is None:
        raise ValueError("invalid sizes")
    return name.decode()


def attend_paged_workspace_bytes(dims: PagedDims) -> int:
    return int(_paged_library().kvc_attend_paged_workspace_bytes(ctypes.byref(dims)))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ints(t: torch.Tensor, name: str, shape, device) -> torch.Tensor:
    if t.dtype == torch.int32 and t.shape == shape and t.device == device and t.is_contiguous():
        return t
    if t.shape != shape or t.dtype not in _INTEGERS:
        raise ValueError(f"{name} must be integers of shape {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype == torch.int64:  # a value past 32 bits stays outside every range
        t = t.clamp(-1, 2**31 - 1)
    return t.to(torch.int32).contiguous()


def _check(packed, key_pool, value_pool, key_scale, value_scale, block_table, cu_seqlens_q,
           seqlens_k, what):
    """The shared contract: types, devices, pool and table shapes. Returns
    (int32 tables, (T, Hq, D), (num_blocks, Hk, block_size, Dv))."""
    q = packed[0][1]
    dtype, dev = q.dtype, q.device
    grad = torch.is_grad_enabled()
    for name, t in packed:
        if t.dim() != 3:
            raise ValueError(f"{name} must be 3-D (tokens, heads, width), got {tuple(t.shape)}")
        if t.dtype != dtype or dtype not in DTYPES:
            raise ValueError(f"{name}: one dtype among float32/bfloat16/float16 is needed")
        if t.device != dev:
            raise ValueError("all tensors must be on one device")
        if grad and t.requires_grad:
            raise ValueError(f"{what} has no gradients: call it under torch.no_grad()")
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on a CUDA device only (no CPU path)")
    pool = key_pool.dtype
    if pool != dtype and pool not in EIGHT_BIT:
        raise ValueError("the pools are of the inputs' dtype, float8_e4m3fn or float8_e5m2")
    for name, t in (("key_pool", key_pool), ("value_pool", value_pool)):
        if t.dim() != 4:
            raise ValueError(f"{name} must be [num_blocks, Hk, block_size, width]")
        if t.dtype != pool or t.device != dev:
            raise ValueError("the pools need one dtype and the inputs' device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    T, Hq, Dq = q.shape
    nb, Hk, bs, D = key_pool.shape
    vb, vh, vs, Dv = value_pool.shape
    if (vb, vh, vs) != (nb, Hk, bs):
        raise ValueError("the pools' blocks, heads and block sizes differ")
    if min(nb, Hk, bs, D, Dv, Hq) < 1 or Hq % Hk:
        raise ValueError("need sizes >= 1 and Hq a multiple of Hk")
    if D > 256 or Dv > 256:
        raise ValueError("widths up to 256 are supported")
    if Dq != D:
        raise ValueError("the query's width is not the key pool's")
    if pool in EIGHT_BIT:
        for name, t in (("key_scale", key_scale), ("value_scale", value_scale)):
            if t is None or t.dtype != torch.float32 or t.shape != (nb, Hk):
                raise ValueError(f"an 8-bit pool needs {name}: float32 [num_blocks, Hk]")
            if t.device != dev or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous on the pool's device")
    elif key_scale is not None or value_scale is not None:
        raise ValueError("key_scale / value_scale go with an 8-bit pool only")
    if block_table.dim() != 2 or min(block_table.shape) < 1:
        raise ValueError("block_table must be [B, max_blocks]")
    B = block_table.shape[0]
    return ((_ints(block_table, "block_table", block_table.shape, dev),
             _ints(cu_seqlens_q, "cu_seqlens_q", (B + 1,), dev),
             _ints(seqlens_k, "seqlens_k", (B,), dev)), (T, Hq, D), (nb, Hk, bs, Dv))


def _raw_stream(index: int) -> int:
    """The current stream's handle (torch.cuda.current_stream() without the
    6 us that its Python object takes)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _on_device(device, call, *args):
    """call(*args, the device's current stream) with that device as the current one."""
    index = device.index
    if index == torch.cuda.current_device():
        return call(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return call(*args, _raw_stream(index))


def _max_q(max_seqlen_q, cu, total_q) -> int:
    if max_seqlen_q is None:  # a device sync
        max_seqlen_q = int((cu[1:] - cu[:-1]).max().item())
    if int(max_seqlen_q) < 0:
        raise ValueError("max_seqlen_q must not be negative")
    return max(int(max_seqlen_q), 1 if total_q else 0)


def _packed(t: torch.Tensor) -> torch.Tensor:
    """t itself when its rows are contiguous and its strides not negative or zero
    by expansion of the width, else a copy."""
    return t if t.stride(2) == 1 or t.shape[2] == 1 else t.contiguous()


def _output(out, shape, like, name):
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if out.shape != shape or out.dtype != like.dtype or out.device != like.device \
            or not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)} of the inputs' dtype and device")
    return out


def _status(status, device):
    if status is not None and not (status.device == device and status.dtype == torch.int32
                                   and status.numel() >= 1):
        raise ValueError("status must be an int32 tensor on the inputs' device")
    return status


def append_rotary_paged(query: torch.Tensor, new_key: torch.Tensor, new_value: torch.Tensor,
                        key_pool: torch.Tensor, value_pool: torch.Tensor,
                        block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                        seqlens_k: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                        key_scale: Optional[torch.Tensor] = None,
                        value_scale: Optional[torch.Tensor] = None, interleaved: bool = False,
                        max_seqlen_q: Optional[int] = None,
                        out_query: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None) -> dict:
    """Append packed new tokens to a paged pool with the rotary position
    embedding applied on the way.

    query [T, Hq, D], new_key [T, Hk, D], new_value [T, Hk, Dv] (any token and
    head strides, e.g. column ranges of one projection); key_pool
    [num_blocks, Hk, block_size, D] / value_pool [..., Dv] are updated in place
    at slots K_b - S_b + t. cos, sin [num_positions, R/2] fp32 turn the first
    R elements of each query and key row by the token's position; pairs are
    (d, d + R/2), or (2d, 2d + 1) when ``interleaved``.

    Pools of the inputs' dtype, or float8_e4m3fn / float8_e5m2 with key_scale /
    value_scale [num_blocks, Hk] fp32 (updated in place: a power of two for
    each block and head, growing when a new token needs it; the block's earlier
    rows are then rounded again).

    Returns {"query": the turned queries [T, Hq, D], "key_pool", "value_pool",
    "key_scale", "value_scale"}. Rows behind the last sequence are not written
    (``out_query`` names the buffer to leave them in). ``max_seqlen_q`` (the
    largest S_b) is read from cu_seqlens_q when not given (a device sync).
    ``status``: an int32 CUDA tensor into which KVC_DEV bits are OR-ed. Sequences
    must write distinct blocks. No gradients (inputs that ask for them are refused).
    """
    (table, cu, kl), (T, Hq, D), (nb, Hk, bs, Dv) = _check(
        (("query", query), ("new_key", new_key), ("new_value", new_value)), key_pool, value_pool,
        key_scale, value_scale, block_table, cu_seqlens_q, seqlens_k, "append_rotary_paged")
    if new_key.shape != (T, Hk, D) or new_value.shape != (T, Hk, Dv):
        raise ValueError(f"new_key / new_value must be {(T, Hk, D)} / {(T, Hk, Dv)}")
    for name, t in (("cos", cos), ("sin", sin)):
        if t.dim() != 2 or t.dtype != torch.float32 or t.shape != cos.shape:
            raise ValueError(f"{name} must be float32 [num_positions, R/2], both alike")
        if t.device != query.device:
            raise ValueError("all tensors must be on one device")
    if 2 * cos.shape[1] > D:
        raise ValueError("the tables turn more elements than a row has")
    lib = _paged_library()
    max_q = _max_q(max_seqlen_q, cu, T)
    q, k, v = (_packed(t) for t in (query, new_key, new_value))
    c, s = cos.contiguous(), sin.contiguous()
    out = _output(out_query, (T, Hq, D), query, "out_query")
    dims = make_paged_dims(table.shape[0], T, max_q, Hq, Hk, D, Dv, nb, bs, table.shape[1],
                           query.dtype, key_pool.dtype)
    st = (ctypes.c_int64 * 6)(*q.stride()[:2], *k.stride()[:2], *v.stride()[:2])
    rc = _on_device(
        query.device, lib.kvc_append_rotary_paged, ctypes.byref(dims), 2 * c.shape[1], c.shape[0],
        1 if interleaved else 0, st, q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(),
        cu.data_ptr(), kl.data_ptr(), c.data_ptr(), s.data_ptr(), key_pool.data_ptr(),
        value_pool.data_ptr(), _ptr(key_scale), _ptr(value_scale), out.data_ptr(),
        _ptr(_status(status, query.device)))
    if rc != 0:
        raise KvcError(rc, status_string(rc))
    return {"query": out, "key_pool": key_pool, "value_pool": value_pool, "key_scale": key_scale,
            "value_scale": value_scale}


def attention_over_paged_cache(q: torch.Tensor, key_pool: torch.Tensor, value_pool: torch.Tensor,
                               block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                               seqlens_k: torch.Tensor, key_scale: Optional[torch.Tensor] = None,
                               value_scale: Optional[torch.Tensor] = None,
                               scale: Optional[float] = None, softcap: Optional[float] = None,
                               alibi_slopes: Optional[torch.Tensor] = None,
                               window: Optional[int] = None, max_seqlen_q: Optional[int] = None,
                               out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Read-only attention of packed queries over a paged pool.

    q [T, Hq, D] (any token and head strides); key_pool [num_blocks, Hk,
    block_size, D] / value_pool [..., Dv] of q's dtype, or in 8 bits with
    key_scale / value_scale [num_blocks, Hk] fp32. Row t of sequence b, at
    position p = K_b - S_b + t, sees the slots j <= p, and with ``window`` only
    j > p - window. Scores are scale * q.k (default 1/sqrt(D)); with ``softcap``
    c, c * tanh(s / c); with ``alibi_slopes`` [Hq] fp32, less slope_h * (p - j).

    Returns out [T, Hq, Dv]; rows behind the last sequence are not written
    (``out`` names the buffer to leave them in). ``workspace``: a uint8 CUDA
    tensor of at least attend_paged_workspace_bytes(...) to use instead of a
    new one (one call at a time). ``max_seqlen_q`` (the largest S_b) is read from
    cu_seqlens_q when not given (a device sync). No gradients (inputs that ask
    for them are refused).
    """
    (table, cu, kl), (T, Hq, D), (nb, Hk, bs, Dv) = _check(
        (("q", q),), key_pool, value_pool, key_scale, value_scale, block_table, cu_seqlens_q,
        seqlens_k, "attention_over_paged_cache")
    scale = default_scale(D) if scale is None else float(scale)
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    softcap = 0.0 if softcap is None else float(softcap)
    if not (softcap >= 0.0 and math.isfinite(softcap)):
        raise ValueError("softcap must be positive and finite (None or 0: no cap)")
    window = 0 if window is None else int(window)
    if window < 0:
        raise ValueError("window must not be negative (None or 0: none)")
    if alibi_slopes is not None:
        if alibi_slopes.dtype != torch.float32 or tuple(alibi_slopes.shape) != (Hq,) or \
                alibi_slopes.device != q.device:
            raise ValueError("alibi_slopes must be float32 [Hq] on q's device")
        alibi_slopes = alibi_slopes.contiguous()
    lib = _paged_library()
    max_q = _max_q(max_seqlen_q, cu, T)
    qq = _packed(q)
    out = _output(out, (T, Hq, Dv), q, "out")
    dims = make_paged_dims(table.shape[0], T, max_q, Hq, Hk, D, Dv, nb, bs, table.shape[1], q.dtype,
                           key_pool.dtype)
    if workspace is None:
        workspace = torch.empty(attend_paged_workspace_bytes(dims), dtype=torch.uint8,
                                device=q.device)
    elif workspace.device != q.device or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    st = (ctypes.c_int64 * 2)(*qq.stride()[:2])
    rc = _on_device(
        q.device, lib.kvc_attend_paged, ctypes.byref(dims), st, qq.data_ptr(), key_pool.data_ptr(),
        value_pool.data_ptr(), _ptr(key_scale), _ptr(value_scale), table.data_ptr(), cu.data_ptr(),
        kl.data_ptr(), scale, softcap, _ptr(alibi_slopes), window, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _ptr(_status(status, q.device)))
    if rc != 0:
        raise KvcError(rc, status_string(rc))
    return out
