"""ctypes binding of libmaskattn (include/maskattn.h), same names as the C ABI.

Argument marshalling only: every step of the computation runs in the CUDA
library.  PyTorch supplies device memory and the current stream.  If the
library cannot be built or loaded, every call raises -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_WORKSPACE, ATTN_ERR_CUDA, \
    ATTN_ERR_TIMEOUT = range(6)
ATTN_F16, ATTN_BF16 = 0, 1
ATTN_MASK_NONE, ATTN_MASK_CAUSAL, ATTN_MASK_SLIDING, ATTN_MASK_BLOCK, \
    ATTN_MASK_SLIDING_FIRST = range(5)

# Every symbol include/maskattn.h declares.
EXPORTS = ("attn_workspace_size", "attn_fwd", "attn_bwd", "attn_bwd_noalloc",
           "attn_get_device_status", "attn_noalloc_get_device_status", "attn_profile_enable",
           "attn_profile_read", "attn_status_string", "attn_paged_plan", "attn_paged_store",
           "attn_paged_workspace_size", "attn_paged_fwd", "attn_rope", "attn_paged8_store",
           "attn_paged8_load", "attn_paged8_workspace_size", "attn_paged8_fwd")


class attn_shape_t(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("Sq", ctypes.c_int), ("Skv", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("flags", ctypes.c_int)]


ATTN_FLAG_COMPENSATED = 1
ATTN_FLAG_SINGLE_PASS = 2


class attn_mask_desc_t(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("window", ctypes.c_int), ("bx", ctypes.c_int),
                ("by", ctypes.c_int), ("block_mask", ctypes.c_void_p),
                ("seqlen_q", ctypes.c_void_p), ("seqlen_k", ctypes.c_void_p),
                ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
                ("total_q", ctypes.c_int), ("total_k", ctypes.c_int),
                ("first", ctypes.c_int)]


class attn_pages_t(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("dtype", ctypes.c_int), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong)]


class attn_rope_desc_t(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("factor", ctypes.c_float), ("turns", ctypes.c_void_p)]


class attn_rope_tensor_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int)] + \
               [(n, ctypes.c_longlong) for n in ("x_batch", "x_head", "x_token", "y_batch",
                                                 "y_head", "y_token")]


ATTN_E4M3, ATTN_I8 = 0, 1


class attn_pages8_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("num_pages", "page_size", "Hkv", "dtype", "code",
                                            "block")] + \
               [(n, ctypes.c_longlong) for n in ("page_stride", "head_stride", "token_stride",
                                                 "scale_page_stride", "scale_head_stride")]


class attn_plan_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "page_size", "num_pages", "max_pages",
                                            "table_stride", "max_tokens")] + \
               [(n, ctypes.c_void_p) for n in ("cached", "fresh", "free_pages", "free_count",
                                               "block_table", "cu_seqlens_q", "seqlen_k",
                                               "free_count_out", "slot_map", "position",
                                               "refused")]


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {attn_status_string(code)}")


_lock = threading.Lock()
_lib = None


def load(build: bool = True) -> ctypes.CDLL:
    """Load libmaskattn.so (building it first when sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build else _build.LIB
            lib = ctypes.CDLL(path)
            vp, sz = ctypes.c_void_p, ctypes.c_size_t
            ps, pm = ctypes.POINTER(attn_shape_t), ctypes.POINTER(attn_mask_desc_t)
            lib.attn_workspace_size.argtypes = [ps, pm, ctypes.POINTER(sz)]
            lib.attn_workspace_size.restype = ctypes.c_int
            lib.attn_fwd.argtypes = [ps, vp, vp, vp, vp, pm, ctypes.c_float, vp, vp, vp, sz, vp]
            lib.attn_fwd.restype = ctypes.c_int
            lib.attn_bwd.argtypes = [ps, vp, vp, vp, vp, vp, vp, vp, pm, ctypes.c_float,
                                     vp, vp, vp, vp, vp, sz, vp]
            lib.attn_bwd.restype = ctypes.c_int
            lib.attn_bwd_noalloc.argtypes = [ps, vp, vp, vp, vp, vp, vp, vp, pm, ctypes.c_float,
                                             vp, vp, vp, vp, vp]
            lib.attn_bwd_noalloc.restype = ctypes.c_int
            lib.attn_get_device_status.argtypes = [vp, vp]
            lib.attn_get_device_status.restype = ctypes.c_int
            lib.attn_noalloc_get_device_status.argtypes = [vp]
            lib.attn_noalloc_get_device_status.restype = ctypes.c_int
            lib.attn_profile_enable.argtypes = [ctypes.c_int]
            lib.attn_profile_enable.restype = ctypes.c_int
            lib.attn_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p),
                                              ctypes.POINTER(ctypes.c_float), ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_int)]
            lib.attn_profile_read.restype = ctypes.c_int
            ll, pp = ctypes.c_longlong, ctypes.POINTER(attn_pages_t)
            lib.attn_paged_plan.argtypes = [ctypes.POINTER(attn_plan_t), vp]
            lib.attn_paged_plan.restype = ctypes.c_int
            lib.attn_paged_store.argtypes = [pp, ctypes.c_int, vp, vp, ll, ll, vp, vp, vp, vp]
            lib.attn_paged_store.restype = ctypes.c_int
            lib.attn_paged_workspace_size.argtypes = [ps, ctypes.POINTER(sz)]
            lib.attn_paged_workspace_size.restype = ctypes.c_int
            lib.attn_paged_fwd.argtypes = [ps, pp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp,
                                           pm, ctypes.c_float, vp, vp, vp, sz, vp]
            lib.attn_paged_fwd.restype = ctypes.c_int
            pr, p8 = ctypes.POINTER(attn_rope_tensor_t), ctypes.POINTER(attn_pages8_t)
            lib.attn_rope.argtypes = [ctypes.POINTER(attn_rope_desc_t), ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, pr, pr, vp, ll, ctypes.c_int, vp]
            lib.attn_rope.restype = ctypes.c_int
            lib.attn_paged8_store.argtypes = [p8, ctypes.c_int, vp, vp, ll, ll, vp, vp, vp, vp, vp,
                                              vp]
            lib.attn_paged8_store.restype = ctypes.c_int
            lib.attn_paged8_load.argtypes = [p8, ctypes.c_int, ctypes.c_int, vp, vp, vp,
                                             ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                             vp]
            lib.attn_paged8_load.restype = ctypes.c_int
            lib.attn_paged8_workspace_size.argtypes = [ps, pm, ctypes.POINTER(sz)]
            lib.attn_paged8_workspace_size.restype = ctypes.c_int
            lib.attn_paged8_fwd.argtypes = [ps, p8, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                            ctypes.c_int, vp, pm, ctypes.c_float, vp, vp, vp, sz,
                                            vp]
            lib.attn_paged8_fwd.restype = ctypes.c_int
            lib.attn_status_string.argtypes = [ctypes.c_int]
            lib.attn_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


# ------------------------------------------------------------------ raw C ABI

def attn_status_string(code: int) -> str:
    return load().attn_status_string(int(code)).decode()


def attn_workspace_size(shape: attn_shape_t, mask: attn_mask_desc_t):
    n = ctypes.c_size_t(0)
    r = load().attn_workspace_size(ctypes.byref(shape), ctypes.byref(mask), ctypes.byref(n))
    return r, n.value


def attn_fwd(shape, q, k, v, sink, mask, scale, o, lse, ws, ws_bytes, stream) -> int:
    return load().attn_fwd(ctypes.byref(shape), q, k, v, sink, ctypes.byref(mask),
                           ctypes.c_float(scale), o, lse, ws, ws_bytes, stream)


def attn_bwd(shape, q, k, v, o, dO, lse, sink, mask, scale, dq, dk, dv, dsink, ws, ws_bytes,
             stream) -> int:
    return load().attn_bwd(ctypes.byref(shape), q, k, v, o, dO, lse, sink, ctypes.byref(mask),
                           ctypes.c_float(scale), dq, dk, dv, dsink, ws, ws_bytes, stream)


def attn_bwd_noalloc(shape, q, k, v, o, dO, lse, sink, mask, scale, dq, dk, dv, dsink,
                     stream) -> int:
    """attn_bwd with the library's fixed device scratch instead of a workspace."""
    return load().attn_bwd_noalloc(ctypes.byref(shape), q, k, v, o, dO, lse, sink,
                                   ctypes.byref(mask), ctypes.c_float(scale), dq, dk, dv, dsink,
                                   stream)


def attn_get_device_status(ws, stream) -> int:
    return load().attn_get_device_status(ws, stream)


def attn_noalloc_get_device_status(stream) -> int:
    """Status word of the last attn_bwd_noalloc call on the current device."""
    return load().attn_noalloc_get_device_status(stream)


def attn_profile_enable(on: bool) -> int:
    return load().attn_profile_enable(1 if on else 0)


def attn_profile_read(capacity: int = 16):
    """[(kernel name, ms)] of the most recent profiled call."""
    names = (ctypes.c_char_p * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = ctypes.c_int(0)
    r = load().attn_profile_read(names, ms, capacity, ctypes.byref(n))
    if r != ATTN_OK:
        raise AttnError(r, "attn_profile_read")
    return [(names[i].decode(), float(ms[i])) for i in range(min(n.value, capacity))]


# ------------------------------------------------------------- torch helpers

def _ints_ptr(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    return t.data_ptr()


@dataclass
class Mask:
    kind: int = ATTN_MASK_NONE
    window: int = 0
    bx: int = 1
    by: int = 1
    block_mask: Optional[torch.Tensor] = None   # uint8 [B,Hq,nQB,nKB] on the device
    seqlen_q: Optional[torch.Tensor] = None     # int32 [B] on the device: valid query rows
    seqlen_k: Optional[torch.Tensor] = None     # int32 [B] on the device: valid keys
    # packed layout: int32 [B + 1] cumulative offsets on the device, the
    # longest lengths (the shape's Sq, Skv) and the tensors' token counts
    cu_seqlens_q: Optional[torch.Tensor] = None
    cu_seqlens_k: Optional[torch.Tensor] = None
    max_seqlen_q: int = 0
    max_seqlen_k: int = 0
    total_q: int = 0
    total_k: int = 0
    first: int = 0   # ATTN_MASK_SLIDING_FIRST: first keys that stay visible

    @property
    def packed(self) -> bool:
        return self.cu_seqlens_q is not None

    def tensors(self):
        return (self.block_mask, self.seqlen_q, self.seqlen_k, self.cu_seqlens_q,
                self.cu_seqlens_k)

    def desc(self) -> attn_mask_desc_t:
        bm = self.block_mask
        return attn_mask_desc_t(self.kind, self.window, self.bx, self.by,
                                None if bm is None else bm.data_ptr(),
                                _ints_ptr(self.seqlen_q, "seqlen_q"),
                                _ints_ptr(self.seqlen_k, "seqlen_k"),
                                _ints_ptr(self.cu_seqlens_q, "cu_seqlens_q"),
                                _ints_ptr(self.cu_seqlens_k, "cu_seqlens_k"), self.total_q,
                                self.total_k, self.first)


def _code_of(dtype: torch.dtype) -> int:
    if dtype == torch.float16:
        return ATTN_F16
    if dtype == torch.bfloat16:
        return ATTN_BF16
    raise TypeError(f"unsupported dtype {dtype}")


def _dtype_code(t: torch.Tensor) -> int:
    return _code_of(t.dtype)


def shape_of(q: torch.Tensor, k: torch.Tensor, flags: int = 0,
             mask: Optional[Mask] = None) -> attn_shape_t:
    """BHSD tensors [B,H,S,D]; or, with a packed mask, token-major [T,H,D]
    tensors whose batch and longest lengths come from the mask."""
    if mask is not None and mask.packed:
        _, Hq, D = q.shape
        _, Hkv, _ = k.shape
        B = mask.cu_seqlens_q.numel() - 1
        return attn_shape_t(B, Hq, Hkv, mask.max_seqlen_q, mask.max_seqlen_k, D, _dtype_code(q),
                            flags)
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    return attn_shape_t(B, Hq, Hkv, Sq, Skv, D, _dtype_code(q), flags)


def packed_mask(kind: int, seqlens_q, seqlens_k, device, window: int = 0, bx: int = 1,
                by: int = 1, block_mask: Optional[torch.Tensor] = None, first: int = 0) -> Mask:
    """Mask for the packed layout from per-sequence lengths (host integers)."""
    import itertools
    lq, lk = [int(x) for x in seqlens_q], [int(x) for x in seqlens_k]
    cq = [0] + list(itertools.accumulate(lq))
    ck = [0] + list(itertools.accumulate(lk))
    return Mask(kind=kind, window=window, bx=bx, by=by, block_mask=block_mask,
                cu_seqlens_q=torch.tensor(cq, dtype=torch.int32, device=device),
                cu_seqlens_k=torch.tensor(ck, dtype=torch.int32, device=device),
                max_seqlen_q=max(lq), max_seqlen_k=max(lk), total_q=cq[-1], total_k=ck[-1],
                first=first)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object (4 us of a call's host time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


_nothing = contextlib.nullcontext()


def _alloc_on(stream):
    """Tensors that a call makes belong to the stream that it runs on: the
    allocator reuses a tensor's memory in the order of its own stream.  A caller
    that uses them on another one calls their record_stream(other) before it
    drops them."""
    return _nothing if stream is None else torch.cuda.stream(stream)


def workspace(shape: attn_shape_t, mask, device) -> torch.Tensor:
    """mask: a Mask, or its desc()."""
    r, n = attn_workspace_size(shape, mask.desc() if isinstance(mask, Mask) else mask)
    if r != ATTN_OK:
        raise AttnError(r, "attn_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _check(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def fwd(q, k, v, sink, mask: Mask, scale: float, ws: Optional[torch.Tensor] = None,
        stream=None):
    """Forward; returns (o, lse), which belong to `stream` where one is given:
    before they are dropped, record_stream tells of every other stream that
    uses them."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    if sink is not None:
        _int_tensor(sink, "sink", q.shape[1], torch.float32)
    shape = shape_of(q, k, mask=mask)
    lse_shape = (q.shape[1], q.shape[0]) if mask.packed else q.shape[:3]   # [Hq, T] when packed
    desc = mask.desc()
    with _alloc_on(stream):
        o = torch.empty_like(q)
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
        if ws is None:
            ws = workspace(shape, desc, q.device)
    with _one_device(q, k, v, sink, ws, *mask.tensors()):
        r = attn_fwd(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(sink), desc, scale, _ptr(o),
                     _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, "attn_fwd")
    return o, lse


def bwd(q, k, v, o, dO, lse, sink, mask: Mask, scale: float, ws: Optional[torch.Tensor] = None,
        out=None, stream=None, compensated: bool = False, single_pass: bool = False):
    """Backward; returns (dq, dk, dv, dsink) (dsink is None without a sink).
    compensated: P and dS enter the contractions as high part + remainder.
    single_pass: dq from partials of the key-stationary kernel, summed by a
    reduction kernel (ATTN_FLAG_SINGLE_PASS) instead of the dq kernel.
    Gradients that are not given in `out` belong to `stream`, as fwd's results
    do."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (lse, "lse")):
        _check(t, n)
    if sink is not None:
        _int_tensor(sink, "sink", q.shape[1], torch.float32)
    flags = (ATTN_FLAG_COMPENSATED if compensated else 0) | \
        (ATTN_FLAG_SINGLE_PASS if single_pass else 0)
    shape = shape_of(q, k, flags, mask=mask)
    desc = mask.desc()
    with _alloc_on(stream if out is None or ws is None else None):
        if out is None:
            dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
            dsink = torch.empty_like(sink) if sink is not None else None
        else:
            dq, dk, dv, dsink = out
        if ws is None:
            ws = workspace(shape, desc, q.device)
    with _one_device(q, k, v, o, dO, lse, sink, dq, dk, dv, dsink, ws, *mask.tensors()):
        r = attn_bwd(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(sink),
                     desc, scale, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dsink), _ptr(ws),
                     ws.numel(), _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, "attn_bwd")
    return dq, dk, dv, dsink


def device_status(ws: torch.Tensor, stream=None) -> int:
    """Status of the last call that used `ws`, after what its device's current
    stream, or `stream`, still has to do."""
    with _one_device(ws):
        return attn_get_device_status(_ptr(ws), _stream(stream))


# ------------------------------------------------------------- rotary positions

def attn_rope(rope: attn_rope_desc_t, dtype, B, S, q, k, position, position_stride, inverse,
              stream) -> int:
    return load().attn_rope(ctypes.byref(rope), dtype, B, S, ctypes.byref(q),
                            None if k is None else ctypes.byref(k), position, position_stride,
                            inverse, stream)


@dataclass
class RopeScaling:
    """Rotary frequencies for contexts `factor` times as long as a model was
    trained on.  kind:
      "linear"  every frequency divided by factor;
      "raised"  the base multiplied by factor^(R / (R - 2)), which divides the
                lowest frequency by factor and keeps the highest (R: rotary_dim);
      "parts"   pairs that turn more than `high` times in original_length
                positions keep their frequency, those that turn less than `low`
                times are divided by factor, the others in between in proportion;
                cos and sin are multiplied by `attention`, without one by
                0.1 ln(factor) + 1."""
    kind: str
    factor: float
    original_length: int = 0
    low: float = 1.0
    high: float = 32.0
    attention: Optional[float] = None


def rope_frequencies(rotary_dim: int, base: float = 10000.0,
                     scaling: Optional[RopeScaling] = None):
    """([rotary_dim / 2] radians a position of each pair, what cos and sin are
    multiplied by): base^(-2 i / rotary_dim), scaled."""
    R = rotary_dim
    if R < 2 or R % 2 or not base > 0:
        raise ValueError("rotary_dim must be even and positive, base positive")
    kind = None if scaling is None else scaling.kind
    if kind not in (None, "linear", "raised", "parts"):
        raise ValueError(f"unknown scaling {kind!r}")
    if scaling is not None and not scaling.factor > 0:
        raise ValueError("the scaling's factor must be positive")
    if kind == "raised":
        if R == 2:
            raise ValueError('"raised" needs more than one pair')
        base = base * scaling.factor ** (R / (R - 2))
    w = [base ** (-2 * i / R) for i in range(R // 2)]
    if kind == "linear":
        w = [x / scaling.factor for x in w]
    factor = 1.0 if kind is None or scaling.attention is None else scaling.attention
    if kind == "parts":
        if scaling.original_length < 1 or not scaling.high > scaling.low:
            raise ValueError('"parts" needs original_length and high > low')
        for i, x in enumerate(w):
            turns = scaling.original_length * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - scaling.low) / (scaling.high - scaling.low)))
            w[i] = x * (keep + (1 - keep) / scaling.factor)
        if scaling.attention is None:
            factor = 0.1 * math.log(scaling.factor) + 1 if scaling.factor > 1 else 1.0
    return w, factor


class Rope:
    """Rotary positions of heads of 128, kept by a program for its models' life:
    the first rotary_dim elements (a multiple of 16) turn, in pairs (i, i +
    rotary_dim / 2), or (2 i, 2 i + 1) if interleaved.  frequencies: radians a
    position of each pair in place of those of base and scaling; factor: what cos
    and sin are multiplied by then."""

    def __init__(self, rotary_dim: int = 128, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[RopeScaling] = None, frequencies=None, factor: float = 1.0,
                 device="cuda"):
        if frequencies is None:
            frequencies, factor = rope_frequencies(rotary_dim, base, scaling)
        elif scaling is not None:
            raise ValueError("frequencies come scaled")
        w = [float(x) for x in frequencies]
        if len(w) != rotary_dim // 2 or not all(math.isfinite(x) for x in w):
            raise ValueError("frequencies must be rotary_dim / 2 finite numbers")
        # 2^64 turns are one: what a negative or a large frequency comes to
        turns = [round(x / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for x in w]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns],
                                  dtype=torch.int64, device=device)
        self.rotary_dim, self.interleaved, self.factor = rotary_dim, bool(interleaved), factor
        self.desc = attn_rope_desc_t(rotary_dim, int(self.interleaved), factor,
                                     self.turns.data_ptr())


def _rope_tensor(x: torch.Tensor, y: torch.Tensor) -> attn_rope_tensor_t:
    xs, ys = x.stride(), y.stride()
    if x.dim() == 3:   # rows [T, heads, 128]
        return attn_rope_tensor_t(x.data_ptr(), y.data_ptr(), x.shape[1], 0, xs[1], xs[0], 0,
                                  ys[1], ys[0])
    return attn_rope_tensor_t(x.data_ptr(), y.data_ptr(), x.shape[1], *xs[:3], *ys[:3])


def rope(rp: Rope, q, k=None, position=None, out=None, stream=None, inverse: bool = False):
    """Queries and keys turned by their positions, packed rows [T, heads, 128] or
    [B, heads, S, 128], possibly slices of wider tensors; returns (q, k).  k may
    be None.  position: int32 [T], or [B, S] or [S]; None: counted from 0 (in
    every sequence).  Rows at a negative position are not written.  out: (q, k) to
    write, which may be the inputs themselves; without it they are contiguous and
    belong to `stream`, as fwd's results do."""
    qs, xs = tuple(q.shape), q.stride()
    rows = len(qs) == 3
    if not (rows or len(qs) == 4) or qs[-1] != 128 or xs[-1] != 1:
        raise ValueError("q must be [T, heads, 128] or [B, heads, S, 128], its last stride 1")
    S, B = (qs[0], 1) if rows else (qs[2], qs[0])
    code = _dtype_code(q)
    if k is not None:
        ks = tuple(k.shape)
        if ks[:1] + ks[2:] != qs[:1] + qs[2:] or k.stride(-1) != 1 or k.dtype != q.dtype:
            raise ValueError("k must have q's type, layout and tokens")
    p_stride = 0
    if position is not None:
        shape = tuple(position.shape)
        if position.dtype != torch.int32 or not position.is_contiguous() or \
                not (shape == (S,) or (shape == (B, S) and not rows)):
            raise ValueError("position must be a contiguous int32 tensor, one a token")
        p_stride = S if len(shape) == 2 else 0
    if out is None:
        with _alloc_on(stream):
            y = torch.empty(qs, dtype=q.dtype, device=q.device)
            z = None if k is None else torch.empty(ks, dtype=q.dtype, device=q.device)
    else:
        y, z = out
        for o, x, n in ((y, q, "q"), (z, k, "k")):
            if (o is None) != (x is None) or (o is not None and (
                    o.shape != x.shape or o.dtype != x.dtype or o.stride(-1) != 1)):
                raise ValueError(f"out's {n} must be like {n}, its last stride 1")
    with _one_device(q, k, position, y, z, rp.turns):
        r = attn_rope(rp.desc, code, B, S, _rope_tensor(q, y),
                      None if k is None else _rope_tensor(k, z), _ptr(position), p_stride,
                      int(inverse), _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, "attn_rope")
    return y, z


def rope_bwd(rp: Rope, dq, dk=None, position=None, out=None, stream=None):
    """The gradients of rope's inputs from those of its outputs, in rope's forms:
    turned back."""
    return rope(rp, dq, dk, position, out, stream, inverse=True)


# ------------------------------------------------------------- paged cache

def attn_paged_plan(plan: attn_plan_t, stream) -> int:
    return load().attn_paged_plan(ctypes.byref(plan), stream)


def attn_paged_store(pages: attn_pages_t, T, k, v, k_stride, v_stride, slot_map, k_pages, v_pages,
                     stream) -> int:
    return load().attn_paged_store(ctypes.byref(pages), T, k, v, k_stride, v_stride, slot_map,
                                   k_pages, v_pages, stream)


def attn_paged_workspace_size(shape: attn_shape_t):
    n = ctypes.c_size_t(0)
    r = load().attn_paged_workspace_size(ctypes.byref(shape), ctypes.byref(n))
    return r, n.value


def attn_paged_fwd(shape, pages, q, k_pages, v_pages, block_table, table_stride, max_pages, sink,
                   mask, scale, o, lse, ws, ws_bytes, stream) -> int:
    return load().attn_paged_fwd(ctypes.byref(shape), ctypes.byref(pages), q, k_pages, v_pages,
                                 block_table, table_stride, max_pages, sink, ctypes.byref(mask),
                                 ctypes.c_float(scale), o, lse, ws, ws_bytes, stream)


def attn_paged8_store(pages: attn_pages8_t, T, k, v, k_stride, v_stride, slot_map, k_pages,
                      v_pages, k_scales, v_scales, stream) -> int:
    return load().attn_paged8_store(ctypes.byref(pages), T, k, v, k_stride, v_stride, slot_map,
                                    k_pages, v_pages, k_scales, v_scales, stream)


def attn_paged8_load(pages: attn_pages8_t, B, total, start, cu_seqlens, block_table, table_stride,
                     max_pages, k_pages, v_pages, k_scales, v_scales, k, v, stream) -> int:
    return load().attn_paged8_load(ctypes.byref(pages), B, total, start, cu_seqlens, block_table,
                                   table_stride, max_pages, k_pages, v_pages, k_scales, v_scales,
                                   k, v, stream)


def attn_paged8_workspace_size(shape: attn_shape_t, mask: Optional[attn_mask_desc_t] = None):
    n = ctypes.c_size_t(0)
    r = load().attn_paged8_workspace_size(ctypes.byref(shape),
                                          None if mask is None else ctypes.byref(mask),
                                          ctypes.byref(n))
    return r, n.value


def attn_paged8_fwd(shape, pages: attn_pages8_t, q, k_pages, v_pages, k_scales, v_scales,
                    block_table, table_stride, max_pages, sink, mask, scale, o, lse, ws, ws_bytes,
                    stream) -> int:
    return load().attn_paged8_fwd(ctypes.byref(shape), ctypes.byref(pages), q, k_pages, v_pages,
                                  k_scales, v_scales, block_table, table_stride, max_pages, sink,
                                  ctypes.byref(mask), scale, o, lse, ws, ws_bytes, stream)


def _one_device(*tensors):
    """All tensors on one CUDA device: a guard that makes it current."""
    devs = {t.get_device() for t in tensors if t is not None}
    dev = devs.pop()
    if devs or dev < 0:   # -1: a tensor of the host
        raise ValueError("every tensor must be a CUDA tensor, all on one device")
    return _nothing if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _int_tensor(t: torch.Tensor, name: str, numel: int, dtype=torch.int32):
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != numel:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel}")


class PagedCache:
    """The pages of a key/value cache: k_pages and v_pages of one shape,
    [pages, Hkv, page_size, 128] (layout "HND") or [pages, page_size, Hkv, 128]
    ("NHD"), possibly slices of a larger tensor, with the same strides."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, layout: str = "HND"):
        if layout not in ("HND", "NHD"):
            raise ValueError(f"unknown layout {layout!r}")
        shape = k_pages.shape
        if len(shape) != 4 or shape[3] != 128 or v_pages.shape != shape:
            raise ValueError("k_pages and v_pages must be [pages, ., ., 128] of one shape")
        if v_pages.dtype != k_pages.dtype or v_pages.device != k_pages.device:
            raise ValueError("k_pages and v_pages must have one type and one device")
        hd, td = (1, 2) if layout == "HND" else (2, 1)
        # a dimension of one element may have any stride
        ks, vs = ([128 if n == 1 else m for n, m in zip(shape, t.stride())]
                  for t in (k_pages, v_pages))
        if ks != vs or ks[3] != 1:
            raise ValueError("k_pages and v_pages must have the same strides, 1 for the last")
        self.k_pages, self.v_pages, self.layout = k_pages, v_pages, layout
        self.num_pages, self.Hkv, self.page_size = shape[0], shape[hd], shape[td]
        self.dtype = k_pages.dtype
        self.desc = attn_pages_t(self.num_pages, self.page_size, self.Hkv, _dtype_code(k_pages),
                                 ks[0], ks[hd], ks[td])

    def pointers(self):
        return self.k_pages.data_ptr(), self.v_pages.data_ptr()


_CODES = {torch.float8_e4m3fn: ATTN_E4M3, torch.int8: ATTN_I8}


def _strides(a: torch.Tensor, b: torch.Tensor, shape, one: int):
    """Strides that a and b share, `one` for dimensions of one element, which may
    have any; None where they differ."""
    s, t = a.stride(), b.stride()
    if s == t and 1 not in shape:
        return s
    s = [one if n == 1 else m for n, m in zip(shape, s)]
    return s if s == [one if n == 1 else m for n, m in zip(shape, t)] else None


class PagedCache8:
    """The pages of a key/value cache held in 8 bits: k_pages and v_pages as in
    PagedCache but of torch.float8_e4m3fn or torch.int8, and k_scales and
    v_scales, uint8 [pages, Hkv, page_size // block], of which each byte s stands
    for the factor 2^(s - 127) of `block` tokens of a head (1, 16, 32 or 64; 255:
    NaN).  dtype: the 16-bit type of the values, torch.bfloat16 or float16."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                 layout: str = "HND"):
        if layout not in ("HND", "NHD"):
            raise ValueError(f"unknown layout {layout!r}")
        shape = tuple(k_pages.shape)
        if len(shape) != 4 or shape[3] != 128 or tuple(v_pages.shape) != shape:
            raise ValueError("k_pages and v_pages must be [pages, ., ., 128] of one shape")
        code = _CODES.get(k_pages.dtype)
        if code is None:
            raise TypeError(f"unsupported type of codes {k_pages.dtype}")
        if v_pages.dtype != k_pages.dtype or not (
                k_pages.get_device() == v_pages.get_device() == k_scales.get_device() ==
                v_scales.get_device()):
            raise ValueError("k_pages and v_pages must have one type, all tensors one device")
        hd, td = (1, 2) if layout == "HND" else (2, 1)
        P, Hkv, ps = shape[0], shape[hd], shape[td]
        per = k_scales.shape[2] if k_scales.dim() == 3 else 0
        if per < 1 or ps % per or k_scales.dtype != torch.uint8 or \
                v_scales.dtype != torch.uint8 or tuple(k_scales.shape) != (P, Hkv, per) or \
                tuple(v_scales.shape) != (P, Hkv, per):
            raise ValueError("the scales must be uint8 [pages, Hkv, page_size // block]")
        ks = _strides(k_pages, v_pages, shape, 128)
        if ks is None or ks[3] != 1:
            raise ValueError("k_pages and v_pages must have the same strides, 1 for the last")
        ss = _strides(k_scales, v_scales, (P, Hkv, per), per)
        if ss is None or (per > 1 and ss[2] != 1):
            raise ValueError("k_scales and v_scales must have the same strides, 1 for the last")
        self.k_pages, self.v_pages, self.layout, self.dtype = k_pages, v_pages, layout, dtype
        self.k_scales, self.v_scales = k_scales, v_scales
        self.num_pages, self.Hkv, self.page_size, self.block = P, Hkv, ps, ps // per
        self.desc = attn_pages8_t(P, ps, Hkv, _code_of(dtype), code, self.block, ks[0], ks[hd],
                                  ks[td], ss[0], ss[1])

    @staticmethod
    def empty(num_pages: int, Hkv: int, page_size: int, block: int = 16,
              codes: torch.dtype = torch.float8_e4m3fn, dtype: torch.dtype = torch.bfloat16,
              layout: str = "HND", device="cuda") -> "PagedCache8":
        """A cache of pages that hold nothing yet."""
        shape = (num_pages, Hkv, page_size, 128) if layout == "HND" else \
            (num_pages, page_size, Hkv, 128)
        if block < 1 or page_size % block:
            raise ValueError("block must divide page_size")
        pages = [torch.empty(shape, dtype=codes, device=device) for _ in range(2)]
        scales = [torch.empty(num_pages, Hkv, page_size // block, dtype=torch.uint8,
                              device=device) for _ in range(2)]
        return PagedCache8(*pages, *scales, dtype, layout)

    def pointers(self):
        return (self.k_pages.data_ptr(), self.v_pages.data_ptr(), self.k_scales.data_ptr(),
                self.v_scales.data_ptr())


@dataclass
class PagedPlan:
    """What attn_paged_plan wrote for one step (all on the device)."""
    cu_seqlens_q: torch.Tensor   # int32 [B + 1]
    seqlen_k: torch.Tensor       # int32 [B]
    free_count: torch.Tensor     # int32 [1]
    slot_map: torch.Tensor       # int64 [max_tokens]
    position: torch.Tensor       # int32 [max_tokens]
    refused: torch.Tensor        # int32 [1]

    @staticmethod
    def empty(B: int, max_tokens: int, device) -> "PagedPlan":
        e = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device=device)
        return PagedPlan(e(B + 1), e(B), e(1), e(max_tokens, torch.int64), e(max_tokens), e(1))


def paged_plan(cached, fresh, free_pages, free_count, block_table, page_size: int,
               max_tokens: int, out: Optional[PagedPlan] = None, stream=None) -> PagedPlan:
    """Pages, slots and offsets of one step from the request lengths cached
    and fresh (int32 [B]); free_pages (int32, one entry per page of the cache)
    and block_table (int32 [B, max_pages]) are updated in place.  out: buffers
    of an earlier plan to write (its seqlen_k may be `cached` and its
    free_count `free_count`); a plan made without it belongs to `stream`, as
    fwd's results do."""
    B = cached.numel()
    for t, n, m in ((cached, "cached", B), (fresh, "fresh", B),
                    (free_pages, "free_pages", free_pages.numel()),
                    (free_count, "free_count", 1)):
        _int_tensor(t, n, m)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [B, max_pages] with rows of stride 1")
    if out is None:
        with _alloc_on(stream):
            out = PagedPlan.empty(B, max_tokens, cached.device)
    else:
        for t, n, m in ((out.cu_seqlens_q, "cu_seqlens_q", B + 1), (out.seqlen_k, "seqlen_k", B),
                        (out.free_count, "out.free_count", 1), (out.refused, "refused", 1),
                        (out.position, "position", max_tokens)):
            _int_tensor(t, n, m)
        _int_tensor(out.slot_map, "slot_map", max_tokens, torch.int64)
    cols = block_table.shape[1]
    plan = attn_plan_t(B, page_size, free_pages.numel(), cols,
                       block_table.stride(0) if B > 1 else cols, max_tokens, cached.data_ptr(),
                       fresh.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(),
                       block_table.data_ptr(), out.cu_seqlens_q.data_ptr(),
                       out.seqlen_k.data_ptr(), out.free_count.data_ptr(),
                       out.slot_map.data_ptr(), out.position.data_ptr(), out.refused.data_ptr())
    with _one_device(cached, fresh, free_pages, free_count, block_table, out.cu_seqlens_q,
                     out.seqlen_k, out.free_count, out.slot_map, out.position, out.refused):
        r = attn_paged_plan(plan, _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, "attn_paged_plan")
    return out


def paged_store(cache, k, v, slot_map, stream=None) -> None:
    """Rows of k and v ([T, Hkv, 128], possibly slices of a larger tensor) into
    their slots of the cache, a PagedCache or PagedCache8 (int64 [T]; negative:
    skipped).  A PagedCache8 wants the rows of each block of tokens consecutive,
    as a plan's slot_map has them; its blocks keep the scale of tokens that are
    taken back until they are stored from their first row again."""
    T = slot_map.numel()
    for t, n in ((k, "k"), (v, "v")):
        if t.dtype != cache.dtype or tuple(t.shape) != (T, cache.Hkv, 128) or \
                t.stride(2) != 1 or (cache.Hkv > 1 and t.stride(1) != 128):
            raise ValueError(f"{n} must be [T, Hkv, 128] of the cache's type, its heads 128 apart")
    _int_tensor(slot_map, "slot_map", T, torch.int64)
    row = cache.Hkv * 128
    if isinstance(cache, PagedCache8):
        with _one_device(cache.k_pages, k, v, slot_map):
            r = attn_paged8_store(cache.desc, T, k.data_ptr(), v.data_ptr(),
                                  k.stride(0) if T > 1 else row, v.stride(0) if T > 1 else row,
                                  slot_map.data_ptr(), *cache.pointers(), _stream(stream))
        if r != ATTN_OK:
            raise AttnError(r, "attn_paged8_store")
        return
    with _one_device(cache.k_pages, k, v, slot_map):
        r = attn_paged_store(cache.desc, T, k.data_ptr(), v.data_ptr(),
                             k.stride(0) if T > 1 else row, v.stride(0) if T > 1 else row,
                             slot_map.data_ptr(), cache.k_pages.data_ptr(),
                             cache.v_pages.data_ptr(), _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, "attn_paged_store")


def paged_load(cache: PagedCache8, block_table, cu_seqlens, total: int, start=None, out=None,
               stream=None):
    """Rows of an 8-bit cache back to 16 bits: (k, v) [total, Hkv, 128], of which
    rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 are request b's positions from
    start[b] on (int32 [B + 1] and [B]; start None: from 0).  Rows of no request
    are not written.  out: (k, v) to write; without it they belong to `stream`, as
    fwd's results do."""
    if not isinstance(cache, PagedCache8):
        raise TypeError("paged_load reads a PagedCache8")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [B, max_pages] with rows of stride 1")
    B, cols = block_table.shape
    _int_tensor(cu_seqlens, "cu_seqlens", B + 1)
    if start is not None:
        _int_tensor(start, "start", B)
    if out is None:
        with _alloc_on(stream):
            k, v = (torch.empty(total, cache.Hkv, 128, dtype=cache.dtype,
                                device=cache.k_pages.device) for _ in range(2))
    else:
        k, v = out
        for t, n in ((k, "k"), (v, "v")):
            if tuple(t.shape) != (total, cache.Hkv, 128) or t.dtype != cache.dtype or \
                    not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous [total, Hkv, 128] tensor of the "
                                 "cache's type")
    with _one_device(cache.k_pages, block_table, cu_seqlens, start, k, v):
        r = attn_paged8_load(cache.desc, B, total, _ptr(start), cu_seqlens.data_ptr(),
                             block_table.data_ptr(), block_table.stride(0) if B > 1 else cols,
                             cols, *cache.pointers(), k.data_ptr(), v.data_ptr(),
                             _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, "attn_paged8_load")
    return k, v


def paged_mask(kind: int, plan: PagedPlan, total_q: int, max_seqlen_q: int, max_seqlen_k: int,
               window: int = 0, first: int = 0) -> Mask:
    """Mask of paged_fwd from a plan's offsets and lengths; total_q: rows of q
    (those past the plan's last token are left alone), max_seqlen_q and
    max_seqlen_k: bounds of the new tokens and keys of a request."""
    return Mask(kind=kind, window=window, first=first, cu_seqlens_q=plan.cu_seqlens_q,
                seqlen_k=plan.seqlen_k, total_q=total_q, max_seqlen_q=max_seqlen_q,
                max_seqlen_k=max_seqlen_k)


def paged_shape(q: torch.Tensor, cache, mask: Mask) -> attn_shape_t:
    return attn_shape_t(mask.seqlen_k.numel(), q.shape[1], cache.Hkv, mask.max_seqlen_q,
                        mask.max_seqlen_k, q.shape[2], _dtype_code(q), 0)


# the most that paged_workspace adds for the 16-bit rows of an 8-bit cache's chunks
PAGED8_ROOM = 2 << 30


@functools.lru_cache(maxsize=256)
def _paged_workspace_bytes(shape, mask, most=0, hook=None):
    """(the least, what is asked for).  mask: what of it the 8-bit cache's workspace depends
    on; most: PAGED8_ROOM; hook: MASKATTN_PAGED8_ROOM, which the library reads."""
    sh = attn_shape_t(*shape, 0)
    size, name = (attn_paged_workspace_size, "attn_paged_workspace_size") if mask is None else \
        (attn_paged8_workspace_size, "attn_paged8_workspace_size")
    r, least = size(sh)
    if r != ATTN_OK:
        raise AttnError(r, name)
    if mask is None:
        return least, least
    kind, window, first, total_q = mask
    _, n = attn_paged8_workspace_size(
        sh, attn_mask_desc_t(kind=kind, window=window, first=first, total_q=total_q))
    return least, n if n - least <= most else least


def paged_workspace(q: torch.Tensor, cache, mask: Mask,
                    shape: Optional[attn_shape_t] = None) -> torch.Tensor:
    """A workspace of paged_fwd.  For a PagedCache8 and chunks with room for the rows
    that they see in 16 bits, up to PAGED8_ROOM bytes; where the allocator has no
    memory for that the least, with which the call takes longer (and differs by
    roundings)."""
    sh = shape or paged_shape(q, cache, mask)
    sizes = (sh.B, sh.Hq, sh.Hkv, sh.Sq, sh.Skv, sh.D, sh.dtype)
    if isinstance(cache, PagedCache8):
        least, n = _paged_workspace_bytes(sizes,
                                          (mask.kind, mask.window, mask.first, mask.total_q),
                                          PAGED8_ROOM, os.environ.get("MASKATTN_PAGED8_ROOM"))
    else:
        least, n = _paged_workspace_bytes(sizes, None)
    if n > least:
        try:
            return torch.empty(n, dtype=torch.uint8, device=q.device)
        except torch.OutOfMemoryError:
            pass
    return torch.empty(least, dtype=torch.uint8, device=q.device)


def paged_fwd(q, cache, block_table, sink, mask: Mask, scale: float,
              ws: Optional[torch.Tensor] = None, out=None, stream=None):
    """Attention of the packed new tokens q [total_q, Hq, 128] over the cache, a
    PagedCache or PagedCache8; returns (o, lse).  out: (o, lse) to write, of which
    lse may be None; without it they belong to `stream`, as fwd's results do.  ws: a
    workspace; without it the call takes paged_workspace's from the allocator, for
    chunks over a PagedCache8 up to PAGED8_ROOM bytes (2 GiB) and the least."""
    cu, lens = mask.cu_seqlens_q, mask.seqlen_k
    if cu is None or lens is None or cu.numel() != lens.numel() + 1:
        raise ValueError("the mask needs cu_seqlens_q [B + 1] and seqlen_k [B]")
    if q.dim() != 3 or q.shape[0] != mask.total_q or not q.is_contiguous():
        raise ValueError("q must be a contiguous [total_q, Hq, 128] tensor")
    T, Hq, _ = q.shape
    dtype, B = q.dtype, lens.numel()
    if dtype != cache.dtype:
        raise ValueError("q and the cache must have one type")
    if block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, max_pages]")
    rows, cols = block_table.shape
    row_stride, col_stride = block_table.stride()
    if rows != B or (cols > 1 and col_stride != 1):
        raise ValueError("block_table must be int32 [B, max_pages] with rows of stride 1")
    if sink is not None:
        _int_tensor(sink, "sink", Hq, torch.float32)
    if out is None:
        with _alloc_on(stream):
            o = torch.empty_like(q)
            lse = torch.empty(Hq, T, dtype=torch.float32, device=q.device)
    else:
        o, lse = out
        if o.shape != q.shape or o.dtype != dtype or not o.is_contiguous():
            raise ValueError("o must be a contiguous tensor like q")
        if lse is not None:
            _int_tensor(lse, "lse", T * Hq, torch.float32)
    shape = paged_shape(q, cache, mask)
    with _one_device(q, cache.k_pages, block_table, sink, cu, lens, o, lse, ws):
        if ws is None:
            with _alloc_on(stream):
                ws = paged_workspace(q, cache, mask, shape)
        call, name = (attn_paged8_fwd, "attn_paged8_fwd") if isinstance(cache, PagedCache8) else \
            (attn_paged_fwd, "attn_paged_fwd")
        r = call(shape, cache.desc, q.data_ptr(), *cache.pointers(), block_table.data_ptr(),
                 row_stride if B > 1 else cols, cols, _ptr(sink), mask.desc(), scale,
                 o.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream))
    if r != ATTN_OK:
        raise AttnError(r, name)
    return o, lse


class HostBackward:
    """Backward from pinned host tensors to pinned host tensors, with the
    host<->device copies overlapped with the kernels.

    The heads of a GQA group are independent of every other group, so the
    call is split into runs of whole key/value heads: `chunks` equal runs, or
    a list of the key/value heads in each run (a short first run shortens the
    copy nothing hides, a short last run the copy out that follows the last
    kernel, and longer runs in between leave fewer grid tails).  Chunk c's
    inputs are copied in on one stream while earlier chunks run attn_bwd and
    their gradients are copied out on another; every chunk is one attn_bwd
    call on pointer offsets into device buffers that are allocated once here
    (the library itself allocates nothing).  Consecutive chunks rotate over
    three compute streams, each with a workspace of its own, so that the SMs
    a chunk leaves idle while its largest key tiles finish take the next
    chunks' work; small chunks also shorten the first copy, which nothing
    hides.  With B > 1 a run of heads is not contiguous across the
    batch, and dSink sums over the batch, so the call is not split
    (chunks = 1).

    __call__ enqueues everything behind the caller's current stream and makes
    that stream wait for the last copy out, so synchronising it covers the
    whole call."""

    def __init__(self, B, Hq, Hkv, Sq, Skv, dtype, mask: Mask, scale: float, has_sink: bool,
                 device, chunks=8, compensated: bool = False):
        self.B, self.Hq, self.Hkv, self.Sq, self.Skv = B, Hq, Hkv, Sq, Skv
        self.dtype, self.mask, self.scale, self.has_sink = dtype, mask, scale, has_sink
        self.device = torch.device(device)
        if isinstance(chunks, int):
            sizes = [Hkv // chunks] * chunks if chunks > 0 and Hkv % chunks == 0 else [Hkv]
        else:
            sizes = [int(x) for x in chunks]
            if any(x <= 0 for x in sizes) or sum(sizes) != Hkv:
                raise ValueError(f"runs of key/value heads {sizes} do not cover the {Hkv} heads")
        if B != 1:
            sizes = [Hkv]
        self.sizes = sizes
        self.chunks = len(sizes)
        self.g = Hq // Hkv
        D = 128
        e = dict(dtype=dtype, device=self.device)
        self.dev = {
            "q": torch.empty(B, Hq, Sq, D, **e), "o": torch.empty(B, Hq, Sq, D, **e),
            "dO": torch.empty(B, Hq, Sq, D, **e), "k": torch.empty(B, Hkv, Skv, D, **e),
            "v": torch.empty(B, Hkv, Skv, D, **e),
            "lse": torch.empty(B, Hq, Sq, dtype=torch.float32, device=self.device),
            "dq": torch.empty(B, Hq, Sq, D, **e), "dk": torch.empty(B, Hkv, Skv, D, **e),
            "dv": torch.empty(B, Hkv, Skv, D, **e),
        }
        if has_sink:
            self.dev["sink"] = torch.empty(Hq, dtype=torch.float32, device=self.device)
            self.dev["dsink"] = torch.empty(Hq, dtype=torch.float32, device=self.device)
        code = ATTN_BF16 if dtype == torch.bfloat16 else ATTN_F16
        flags = ATTN_FLAG_COMPENSATED if compensated else 0
        self.cshapes = [attn_shape_t(B, self.g * kv, kv, Sq, Skv, D, code, flags) for kv in sizes]
        nws = min(3, self.chunks)
        # each workspace is sized for whichever run needs most, so any run may use
        # it (with first keys a short run may need more than a long one)
        need = 256
        for shape in self.cshapes:
            r, n = attn_workspace_size(shape, mask.desc())
            if r != ATTN_OK:
                raise AttnError(r, "attn_workspace_size")
            need = max(need, n)
        self.ws = [torch.empty(need, dtype=torch.uint8, device=self.device) for _ in range(nws)]
        self.s_comp = [torch.cuda.Stream(self.device) for _ in range(nws)]
        self.s_in = torch.cuda.Stream(self.device)
        self.s_out = torch.cuda.Stream(self.device)
        self.ev_in = [torch.cuda.Event() for _ in range(self.chunks)]
        self.ev_done = [torch.cuda.Event() for _ in range(self.chunks)]
        self.ev_start = torch.cuda.Event()
        self.ev_out = torch.cuda.Event()
        self.ev_comp = [torch.cuda.Event() for _ in range(len(self.s_comp))]

    def bytes_per_call(self, host_in, host_out):
        h2d = sum(t.numel() * t.element_size() for t in host_in.values() if t is not None)
        d2h = sum(t.numel() * t.element_size() for t in host_out if t is not None)
        return h2d, d2h

    def __call__(self, host_in: dict, host_out):
        """host_in: pinned q, k, v, o, dO, lse (and sink); host_out: pinned
        (dq, dk, dv, dsink)."""
        cur = torch.cuda.current_stream(self.device)
        self.ev_start.record(cur)
        self.s_in.wait_event(self.ev_start)
        for sc in self.s_comp:
            sc.wait_event(self.ev_start)
        g = self.g
        d = self.dev
        k_lo = 0
        for c, kv in enumerate(self.sizes):
            ks = slice(k_lo, k_lo + kv)
            qs = slice(k_lo * g, (k_lo + kv) * g)
            k_lo += kv
            with torch.cuda.stream(self.s_in):
                for n in ("q", "o", "dO", "lse"):
                    d[n][:, qs].copy_(host_in[n][:, qs], non_blocking=True)
                for n in ("k", "v"):
                    d[n][:, ks].copy_(host_in[n][:, ks], non_blocking=True)
                if self.has_sink:
                    d["sink"][qs].copy_(host_in["sink"][qs], non_blocking=True)
                self.ev_in[c].record(self.s_in)
            sc = self.s_comp[c % len(self.s_comp)]
            ws = self.ws[c % len(self.ws)]
            sc.wait_event(self.ev_in[c])
            mask = self.mask
            if mask.block_mask is not None:
                mask = Mask(mask.kind, mask.window, mask.bx, mask.by, mask.block_mask[:, qs],
                            mask.seqlen_q, mask.seqlen_k)
            sink = d["sink"][qs] if self.has_sink else None
            dsink = d["dsink"][qs] if self.has_sink else None
            r = attn_bwd(self.cshapes[c], _ptr(d["q"][:, qs]), _ptr(d["k"][:, ks]),
                         _ptr(d["v"][:, ks]), _ptr(d["o"][:, qs]), _ptr(d["dO"][:, qs]),
                         _ptr(d["lse"][:, qs]), _ptr(sink), mask.desc(), self.scale,
                         _ptr(d["dq"][:, qs]), _ptr(d["dk"][:, ks]), _ptr(d["dv"][:, ks]),
                         _ptr(dsink), _ptr(ws), ws.numel(), _stream(sc))
            if r != ATTN_OK:
                raise AttnError(r, "attn_bwd")
            self.ev_done[c].record(sc)
            self.s_out.wait_event(self.ev_done[c])
            with torch.cuda.stream(self.s_out):
                dq, dk, dv, dsink_h = host_out
                dq[:, qs].copy_(d["dq"][:, qs], non_blocking=True)
                dk[:, ks].copy_(d["dk"][:, ks], non_blocking=True)
                dv[:, ks].copy_(d["dv"][:, ks], non_blocking=True)
                if self.has_sink:
                    dsink_h[qs].copy_(d["dsink"][qs], non_blocking=True)
        self.ev_out.record(self.s_out)
        cur.wait_event(self.ev_out)
        # the compute streams are idle once the last copy out has begun; keep
        # the caller's stream ordered after them too (nothing is pending)
        for sc, ev in zip(self.s_comp, self.ev_comp):
            ev.record(sc)
            cur.wait_event(ev)
