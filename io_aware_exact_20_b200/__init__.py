"""Exact (FlashAttention-style) softmax attention for B200 / sm_100a.

A thin Python binding over the C ABI declared in ``include/fa.h`` and
implemented by ``libfa_b200.so`` (built in this directory by
``io_aware_exact_20_b200.build``).  The binding only marshals arguments:
PyTorch supplies device memory and the current stream; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or the tensors are not on a CUDA device, the call raises.

Entry points mirror the C names: ``fa_fwd`` / ``fa_bwd`` take raw pointers
exactly like the C functions; ``forward`` / ``backward`` wrap them for torch
tensors of layout [B, H, N, d].
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct

from .build import LIB_PATH

__all__ = [
    "FaError", "library", "forward", "backward", "backward_phases", "bwd_workspace_size",
    "forward_general", "backward_general", "general_workspace_size",
    "merge_partial", "accumulate_bf16", "convert_f32_bf16", "qkv_projection",
    "dropout_mask", "last_device_status", "set_wait_timeout_ns", "set_block_mask_bitmap",
    "wait_timeout_probe", "set_nvtx", "STATUS", "PagedCache",
]

STATUS = {
    0: "FA_OK",
    1: "FA_ERR_INVALID_ARG",
    2: "FA_ERR_UNSUPPORTED",
    3: "FA_ERR_CUDA",
    4: "FA_ERR_TIMEOUT",
    5: "FA_ERR_WORKSPACE",
    6: "FA_ERR_BOUNDS",
}


# NVTX ranges around the entry points below, for timeline profilers: off unless
# FA_NVTX is set to a non-zero value or set_nvtx(True) is called.
_NVTX = os.environ.get("FA_NVTX", "0") not in ("", "0")


def set_nvtx(enabled):
    """Marks each call of the entry points with an NVTX range ("fa.forward",
    "fa.backward", ...) when enabled."""
    global _NVTX
    _NVTX = bool(enabled)


def _nvtx(name):
    def deco(fn):
        @functools.wraps(fn)
        def wrapped(*args, **kwargs):
            if not _NVTX:
                return fn(*args, **kwargs)
            import torch
            torch.cuda.nvtx.range_push(name)
            try:
                return fn(*args, **kwargs)
            finally:
                torch.cuda.nvtx.range_pop()
        return wrapped
    return deco


class FaError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


_LIB = None
_vp, _i, _f, _u64, _sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                          ctypes.c_uint64, ctypes.c_size_t)

class Strides(ctypes.Structure):
    """fa_strides_t: element strides of a [batch, head, row, d] view."""
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("row", ctypes.c_int64)]


class AttentionDesc(ctypes.Structure):
    """fa_attention_desc_t (include/fa.h), field for field."""
    _fields_ = [
        ("batch", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("seqlen_q", ctypes.c_int), ("seqlen_k", ctypes.c_int),
        ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("total_q", ctypes.c_int), ("total_k", ctypes.c_int),
        ("seqlens_k", ctypes.c_void_p),
        ("softmax_scale", ctypes.c_float), ("causal", ctypes.c_int),
        ("dropout_p", ctypes.c_float), ("seed", ctypes.c_uint64),
        ("block_mask", ctypes.c_void_p),
        ("q", Strides), ("k", Strides), ("v", Strides), ("o", Strides), ("dout", Strides),
        ("dq", Strides), ("dk", Strides), ("dv", Strides),
        ("dropout_row0", ctypes.c_int64), ("dropout_key0", ctypes.c_int64),
        ("heads_kv", ctypes.c_int),
        ("window", ctypes.c_int), ("sinks", ctypes.c_int),
    ]


class CacheDesc(ctypes.Structure):
    """fa_cache_t (include/fa.h), field for field."""
    _fields_ = [
        ("layers", ctypes.c_int), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("slots", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_layer", ctypes.c_int64), ("v_layer", ctypes.c_int64),
        ("ks", Strides), ("vs", Strides),
        ("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("refs", ctypes.c_void_p),
    ]


# AttentionDesc's fields in order, with native alignment
_DESC_CODES = "iiiii" "PP" "ii" "P" "f" "i" "f" "Q" "P" + "q" * 24 + "qq" "iii"
_DESC = struct.Struct(f"@{_DESC_CODES}0q")


def _pack(*values):
    """An AttentionDesc's bytes.  What a field's type cannot hold becomes what the
    library refuses there: an infinite scale or probability, a size of -1."""
    try:
        return _DESC.pack(*values)
    except (OverflowError, struct.error):
        bits = {"i": 31, "q": 63}
        return _DESC.pack(*(ctypes.c_float(float(x)).value if c == "f"
                            else -1 if c in bits and not -(1 << bits[c]) <= x < 1 << bits[c] else x
                            for c, x in zip(_DESC_CODES, values)))


_DP = ctypes.POINTER(AttentionDesc)
_CP = ctypes.POINTER(CacheDesc)
_i64 = ctypes.c_int64

# name -> (restype, argtypes); must match include/fa.h
SIGNATURES = {
    "fa_fwd_ex": (_i, [_DP, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fa_bwd_ex_workspace_size": (_sz, [_DP]),
    "fa_bwd_ex": (_i, [_DP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _f, _u64, _vp, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp,
                    _f, _u64, _vp, _vp, _sz, _vp]),
    "fa_bwd_prepare": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _sz, _vp]),
    "fa_bwd_main": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _f, _u64,
                         _vp, _vp, _sz, _vp]),
    "fa_bwd_finish": (_i, [_vp, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i,
                            _vp, _f, _u64, _vp, _vp]),
    "fa_qkv_projection": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "fa_merge_partial": (_i, [_vp, _vp, _vp, _vp, ctypes.c_int64, _i, _vp]),
    "fa_accumulate_bf16": (_i, [_vp, _vp, ctypes.c_int64, _vp]),
    "fa_convert_f32_bf16": (_i, [_vp, _vp, ctypes.c_int64, _vp]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_last_device_status": (_i, [_vp]),
    "fa_set_wait_timeout_ns": (None, [_u64]),
    "fa_debug_dropout_mask": (_i, [_vp, _i, _i, _i, _f, _u64, _vp]),
    "fa_debug_wait_timeout": (_i, [_vp]),
    "fa_debug_set_block_mask_bitmap": (None, [_i]),
    "fa_debug_bounds_checking": (_i, []),
    "fa_debug_set_gqa_split": (None, [_i]),
    "fa_cache_workspace_size": (_sz, [_CP, _i]),
    "fa_cache_extend_workspace_size": (_sz, [_CP, _i]),
    "fa_cache_fork_workspace_size": (_sz, [_CP, _i]),
    "fa_cache_compact_workspace_size": (_sz, [_CP]),
    "fa_cache_copy_pages_workspace_size": (_sz, [_CP, _i]),
    "fa_cache_extend": (_i, [_CP, _vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "fa_cache_write": (_i, [_CP, _i, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i, _i, _vp]),
    "fa_cache_fork": (_i, [_CP, _vp, _vp, _i, _vp, _sz, _vp]),
    "fa_cache_free": (_i, [_CP, _vp, _i, _vp]),
    "fa_cache_compact": (_i, [_CP, _vp, _vp, _sz, _vp]),
    "fa_cache_copy_pages": (_i, [_CP, _CP, _vp, _vp, _i, _vp, _sz, _vp]),
    "fa_cache_attend_workspace_size": (_sz, [_CP, _i, _i, _i, _i]),
    "fa_cache_attend": (_i, [_CP, _i, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i, _i, _f, _i,
                             _i, _vp, _sz, _vp]),
}


def library():
    """The loaded C library (raises if it has not been built).  The
    environment variable FA_B200_LIBRARY may name another build of it (one of
    the checking variants of `build.build_variant`)."""
    global _LIB
    if _LIB is None:
        path = os.environ.get("FA_B200_LIBRARY") or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m io_aware_exact_20_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(code, where):
    if code != 0:
        raise FaError(code, where)


def _stream_ptr(device):
    """The current stream's handle on `device` (a torch.device, an index or None)."""
    import torch
    index = getattr(device, "index", device)
    if index is None:
        return torch.cuda.current_stream(device).cuda_stream
    # the same handle without a Stream object around it (0.1 us for 2 us)
    return torch._C._cuda_getCurrentRawStream(index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_qkv(*ts):
    import torch
    ref = ts[0]
    if ref.dim() != 4:
        raise ValueError("tensors must be [B, H, N, d]")
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if t.dtype != torch.bfloat16:
            raise ValueError("tensors must be bfloat16")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [B, H, N, d]")
        if t.shape != ref.shape or t.device != ref.device:
            raise ValueError("q, k, v (and o, dout) must share shape and device")


def _array(x, dtype, device):
    """x (a tensor, an array or a list) as a contiguous tensor on the device."""
    import torch
    if isinstance(x, torch.Tensor) and x.dtype is dtype and x.device == device and x.is_contiguous():
        return x
    return torch.as_tensor(x, dtype=dtype, device=device).contiguous()


def _masks(seqlens, block_mask, device):
    if seqlens is None and block_mask is None:
        return None, None
    import torch
    return (None if seqlens is None else _array(seqlens, torch.int32, device),
            None if block_mask is None else _array(block_mask, torch.uint8, device))


@_nvtx("fa.forward")
def forward(q, k, v, scale=None, causal=False, seqlens=None, dropout_p=0.0, seed=0,
            block_mask=None, out=None, lse=None):
    """O, LSE = attention(q, k, v) for bf16 CUDA tensors [B, H, N, d]."""
    import torch
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    sl, bm = _masks(seqlens, block_mask, q.device)
    code = library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                            float(scale), int(bool(causal)), _ptr(sl), float(dropout_p),
                            int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(bm), _stream_ptr(q.device))
    _check(code, "fa_fwd")
    return out, lse


def bwd_workspace_size(B, H, N, d):
    return int(library().fa_bwd_workspace_size(B, H, N, d))


@_nvtx("fa.backward")
def backward(q, k, v, o, lse, dout, scale=None, causal=False, seqlens=None, dropout_p=0.0,
             seed=0, block_mask=None, workspace=None, dq=None, dk=None, dv=None):
    """dQ, dK, dV of attention for bf16 CUDA tensors [B, H, N, d]."""
    import torch
    _check_qkv(q, k, v, o, dout)
    B, H, N, d = q.shape
    if scale is None:
        scale = d ** -0.5
    need = bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    sl, bm = _masks(seqlens, block_mask, q.device)
    code = library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                            _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                            int(bool(causal)), _ptr(sl), float(dropout_p),
                            int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(bm), _ptr(workspace),
                            workspace.numel() * workspace.element_size(),
                            _stream_ptr(q.device))
    _check(code, "fa_bwd")
    return dq, dk, dv


@_nvtx("fa.backward_phases")
def backward_phases(q, k, v, o, lse, dout, scale=None, causal=False, seqlens=None,
                    dropout_p=0.0, seed=0, block_mask=None, workspace=None, dq=None, dk=None,
                    dv=None):
    """The three launches of ``backward`` as three callables (prepare, main,
    finish) bound to the same buffers, plus the outputs: lets a caller put
    events or other work between them."""
    import torch
    _check_qkv(q, k, v, o, dout)
    B, H, N, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(bwd_workspace_size(B, H, N, d), dtype=torch.uint8,
                                device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    sl, bm = _masks(seqlens, block_mask, q.device)
    ws, nws = _ptr(workspace), workspace.numel() * workspace.element_size()
    lib = library()
    seed = int(seed) & 0xFFFFFFFFFFFFFFFF

    def prepare():
        _check(lib.fa_bwd_prepare(_ptr(o), _ptr(lse), _ptr(dout), B, H, N, d, ws, nws,
                                  _stream_ptr(q.device)), "fa_bwd_prepare")

    def main():
        _check(lib.fa_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dk), _ptr(dv), B, H,
                               N, d, float(scale), int(bool(causal)), _ptr(sl),
                               float(dropout_p), seed, _ptr(bm), ws, nws,
                               _stream_ptr(q.device)), "fa_bwd_main")

    def finish():
        _check(lib.fa_bwd_finish(_ptr(dq), B, H, N, d, float(scale), ws, nws,
                                 _stream_ptr(q.device)), "fa_bwd_finish")

    return (prepare, main, finish), (dq, dk, dv), (sl, bm, workspace)


def dropout_mask(B, H, N, dropout_p, seed, device="cuda"):
    """Keep bits [B, H, N, N] (uint8) from the library's device generator."""
    import torch
    keep = torch.empty((B, H, N, N), dtype=torch.uint8, device=device)
    code = library().fa_debug_dropout_mask(_ptr(keep), B, H, N, float(dropout_p),
                                           int(seed) & 0xFFFFFFFFFFFFFFFF,
                                           _stream_ptr(keep.device))
    _check(code, "fa_debug_dropout_mask")
    return keep


def last_device_status(device=None):
    import torch
    return library().fa_last_device_status(_stream_ptr(device or torch.cuda.current_device()))


def set_wait_timeout_ns(ns):
    library().fa_set_wait_timeout_ns(int(ns))


def set_gqa_split(parts):
    """Test support: parts per backward unit under grouped K / V heads (0 =
    chosen from the problem's size; ignored unless it divides the group)."""
    library().fa_debug_set_gqa_split(int(parts))


def set_block_mask_bitmap(enabled):
    """Test support: False makes later launches walk block masks byte by byte."""
    library().fa_debug_set_block_mask_bitmap(1 if enabled else 0)


def wait_timeout_probe(device=None):
    import torch
    _check(library().fa_debug_wait_timeout(_stream_ptr(device or torch.cuda.current_device())),
           "fa_debug_wait_timeout")


# ---------------------------------------------------------------------------
# general layouts: [B, H, N, d] / [B, N, H, d] with any strides, packed
# variable-length batches [T, H, d], N_q != N_k, d in {32, 64, 96, 128}
# ---------------------------------------------------------------------------

def _strides(t, layout):
    """Element strides (batch, head, row) of a tensor in the layout."""
    s = t.stride()
    if s[-1] != 1:
        raise ValueError("the head dimension must be contiguous")
    if layout == "bhsd":
        return s[:3]
    if layout == "bshd":
        return s[0], s[2], s[1]
    return 0, s[1], s[0]


def _dims(t, layout):
    """(batch, rows, heads, d) of a tensor in the given layout."""
    if layout == "bhsd":
        return t.shape[0], t.shape[2], t.shape[1], t.shape[3]
    if layout == "bshd":
        return t.shape[0], t.shape[1], t.shape[2], t.shape[3]
    return None, t.shape[0], t.shape[1], t.shape[2]


# the tensors of a call that have Q's shape; the others (k, v, dk, dv) have K's
_Q_SIDE = ("q", "o", "dout", "dq")
_UNUSED = (0, 0, 0)


def _desc(q, k, layout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, causal,
          seqlens_k, dropout_p, seed, block_mask, tensors, dropout_pos=(0, 0), window=0,
          sinks=0):
    import torch
    if layout not in ("bhsd", "bshd", "thd"):
        raise ValueError(f"unknown layout {layout!r}")
    want_dim = 3 if layout == "thd" else 4
    device, index, bf16, shape_q, shape_k = q.device, q.get_device(), torch.bfloat16, q.shape, k.shape
    for name, t in tensors.items():
        shape, ref = t.shape, shape_q if name in _Q_SIDE else shape_k
        if len(shape) != want_dim:
            raise ValueError(f"{name}: a {want_dim}-D tensor is expected for layout {layout!r}")
        if index < 0 or t.get_device() != index or t.dtype is not bf16:
            raise ValueError(f"{name}: bfloat16 on the device of q is expected")
        if shape != ref:
            raise ValueError(f"{name}: shape {tuple(shape)} differs from "
                             f"{'q' if name in _Q_SIDE else 'k'} {tuple(ref)}")
    Bq, Nq, H, d = _dims(q, layout)
    Bk, Nk, Hk, dk = _dims(k, layout)
    if d != dk or Hk < 1 or H % Hk:
        raise ValueError("q and k must have the same head dim, and q's heads must be a multiple "
                         "of k's (grouped-query attention)")
    cq = ck = None
    if layout == "thd":
        if cu_seqlens_q is None or cu_seqlens_k is None:
            raise ValueError("the packed layout needs cu_seqlens_q and cu_seqlens_k")
        if max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("the packed layout needs max_seqlen_q and max_seqlen_k")
        cq = _array(cu_seqlens_q, torch.int32, device)
        ck = cq if cu_seqlens_k is cu_seqlens_q else _array(cu_seqlens_k, torch.int32, device)
        sizes = (cq.numel() - 1, H, d, int(max_seqlen_q), int(max_seqlen_k), cq.data_ptr(),
                 ck.data_ptr(), Nq, Nk)
    else:
        if Bq != Bk:
            raise ValueError("q and k must have the same batch size")
        sizes = (Bq, H, d, Nq, Nk, 0, 0, 0, 0)
    sl, bm = _masks(seqlens_k, block_mask, device)
    get = {name: _strides(t, layout) for name, t in tensors.items()}.get
    # all fields at once (4 us less than one by one)
    a = AttentionDesc.from_buffer_copy(_pack(
        *sizes, _ptr(sl) or 0, d ** -0.5 if scale is None else scale, bool(causal), dropout_p,
        int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(bm) or 0, *get("q", _UNUSED), *get("k", _UNUSED),
        *get("v", _UNUSED), *get("o", _UNUSED), *get("dout", _UNUSED), *get("dq", _UNUSED),
        *get("dk", _UNUSED), *get("dv", _UNUSED), int(dropout_pos[0]), int(dropout_pos[1]), Hk,
        *_window(window, sinks)))
    return a, (cq, ck, sl, bm)


def _window(window, sinks):
    """(window, sinks) as C ints; past 2^31 - 1 a window hides nothing (the
    library takes one as long as the keys for none)."""
    window, sinks = int(window or 0), int(sinks or 0)
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    return min(window, 2**31 - 1), min(sinks, 2**31 - 1)


@_nvtx("fa.forward_general")
def forward_general(q, k, v, *, layout="bhsd", cu_seqlens_q=None, cu_seqlens_k=None,
                    max_seqlen_q=None, max_seqlen_k=None, scale=None, causal=False,
                    seqlens_k=None, dropout_p=0.0, seed=0, block_mask=None, out=None, lse=None,
                    dropout_row0=0, dropout_key0=0, window=0, sinks=0):
    """O, LSE for a general layout (fa_fwd_ex).

    layout "bhsd": q [B, H, N_q, d], k / v [B, H, N_k, d]; "bshd": q [B, N_q, H, d],
    k / v [B, N_k, H, d]; "thd": packed q [T_q, H, d], k / v [T_k, H, d] with int32
    offsets cu_seqlens_q / cu_seqlens_k ([B + 1]) and the longest lengths.  Any
    strides with d contiguous (multiples of 8 elements).  The causal mask is
    bottom-right aligned per sequence.  LSE: [B, H, N_q] or [H, T_q] (packed).
    k and v may have fewer heads than q, a divisor of them (grouped-query
    attention: query head h reads K / V head h // (H / H_kv)).
    dropout_row0 / dropout_key0: positions of the call's first query row and
    first key in the sequence the dropout bits are keyed by (a block of a
    longer sequence); the key position a multiple of 8.
    window (with causal): each query sees the last `window` keys up to its own
    position and the first `sinks` keys of its sequence; 0 or None: all keys.
    """
    import torch
    if out is None:
        out = torch.empty_like(q)
    a, keep = _desc(q, k, layout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale,
                    causal, seqlens_k, dropout_p, seed, block_mask,
                    dict(q=q, k=k, v=v, o=out), (dropout_row0, dropout_key0), window, sinks)
    if lse is None:
        lse = q.new_empty(_lse_shape(q, layout), dtype=torch.float32)
    else:
        _check_lse(lse, q, layout)
    code = library().fa_fwd_ex(ctypes.byref(a), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                               out.data_ptr(), lse.data_ptr(), _stream_ptr(q.device))
    _check(code, "fa_fwd_ex")
    del keep
    return out, lse


def _lse_shape(q, layout):
    """[B, H, N_q] (padded layouts) or [H, T_q] (packed)."""
    if layout == "thd":
        return (q.shape[1], q.shape[0])
    B, Nq, H, _ = _dims(q, layout)
    return (B, H, Nq)


def _check_lse(lse, q, layout):
    import torch
    shape = _lse_shape(q, layout)
    if (lse.dtype != torch.float32 or lse.device != q.device or tuple(lse.shape) != shape
            or not lse.is_contiguous()):
        raise ValueError(f"lse: contiguous float32 {shape} on the device of q is expected")


def general_workspace_size(q, k, **kw):
    """Workspace bytes of backward_general for these tensors and options."""
    a, keep = _desc(q, k, kw.get("layout", "bhsd"), kw.get("cu_seqlens_q"),
                    kw.get("cu_seqlens_k"), kw.get("max_seqlen_q"), kw.get("max_seqlen_k"),
                    kw.get("scale"), kw.get("causal", False), kw.get("seqlens_k"),
                    kw.get("dropout_p", 0.0), kw.get("seed", 0), kw.get("block_mask"),
                    dict(q=q, k=k, v=k, o=q, dout=q, dq=q, dk=k, dv=k),
                    window=kw.get("window", 0), sinks=kw.get("sinks", 0))
    return int(library().fa_bwd_ex_workspace_size(ctypes.byref(a)))


@_nvtx("fa.backward_general")
def backward_general(q, k, v, o, lse, dout, *, layout="bhsd", cu_seqlens_q=None,
                     cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None, scale=None,
                     causal=False, seqlens_k=None, dropout_p=0.0, seed=0, block_mask=None,
                     workspace=None, dq=None, dk=None, dv=None, dropout_row0=0, dropout_key0=0,
                     window=0, sinks=0):
    """dQ, dK, dV for a general layout (fa_bwd_ex); arguments as forward_general."""
    import torch
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    a, keep = _desc(q, k, layout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale,
                    causal, seqlens_k, dropout_p, seed, block_mask,
                    dict(q=q, k=k, v=v, o=o, dout=dout, dq=dq, dk=dk, dv=dv),
                    (dropout_row0, dropout_key0), window, sinks)
    _check_lse(lse, q, layout)
    lib = library()
    need = int(lib.fa_bwd_ex_workspace_size(ctypes.byref(a)))
    if workspace is None:
        nbytes = max((need + 3) // 4, 1) * 4
        workspace = lse.new_empty(nbytes // 4)
    elif not workspace.is_cuda or workspace.device != q.device:
        raise ValueError("workspace: a tensor on the device of q is expected")
    else:
        nbytes = workspace.numel() * workspace.element_size()
    code = lib.fa_bwd_ex(ctypes.byref(a), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                         lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                         dv.data_ptr(), workspace.data_ptr(), nbytes, _stream_ptr(q.device))
    _check(code, "fa_bwd_ex")
    del keep
    return dq, dk, dv


# ---------------------------------------------------------------------------
# combining partial results (context-parallel attention)
# ---------------------------------------------------------------------------

@_nvtx("fa.merge_partial")
def merge_partial(o_acc, lse_acc, o_part, lse_part):
    """o_acc (fp32 [..., d]), lse_acc (fp32 [...]) <- merge with the partial
    result o_part (bf16 [..., d]), lse_part (fp32 [...]); in place."""
    import torch
    for t, dt in ((o_acc, torch.float32), (lse_acc, torch.float32), (o_part, torch.bfloat16),
                  (lse_part, torch.float32)):
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError("merge_partial: contiguous CUDA tensors of the documented dtypes")
    d = o_acc.shape[-1]
    rows = o_acc.numel() // d
    if o_part.numel() != o_acc.numel() or lse_acc.numel() != rows or lse_part.numel() != rows:
        raise ValueError("merge_partial: shapes differ")
    _check(library().fa_merge_partial(_ptr(o_acc), _ptr(lse_acc), _ptr(o_part), _ptr(lse_part),
                                      rows, d, _stream_ptr(o_acc.device)), "fa_merge_partial")


@_nvtx("fa.accumulate_bf16")
def accumulate_bf16(acc, part):
    """acc (fp32) += part (bf16), elementwise, in place."""
    import torch
    if acc.dtype != torch.float32 or part.dtype != torch.bfloat16 or acc.numel() != part.numel():
        raise ValueError("accumulate_bf16: fp32 accumulator and bf16 part of one size")
    if not (acc.is_cuda and part.is_cuda and acc.is_contiguous() and part.is_contiguous()):
        raise ValueError("accumulate_bf16: contiguous CUDA tensors")
    _check(library().fa_accumulate_bf16(_ptr(acc), _ptr(part), acc.numel(),
                                        _stream_ptr(acc.device)), "fa_accumulate_bf16")


@_nvtx("fa.convert_f32_bf16")
def convert_f32_bf16(src, out=None):
    """bf16 copy of an fp32 tensor (round to nearest even)."""
    import torch
    if src.dtype != torch.float32 or not src.is_cuda or not src.is_contiguous():
        raise ValueError("convert_f32_bf16: a contiguous fp32 CUDA tensor")
    out = torch.empty(src.shape, dtype=torch.bfloat16, device=src.device) if out is None else out
    _check(library().fa_convert_f32_bf16(_ptr(out), _ptr(src), src.numel(),
                                         _stream_ptr(src.device)), "fa_convert_f32_bf16")
    return out


# ---------------------------------------------------------------------------
# fused QKV projection
# ---------------------------------------------------------------------------

@_nvtx("fa.qkv_projection")
def qkv_projection(x, weight, bias, batch, heads, head_dim, q=None, k=None, v=None):
    """Q, K, V [B, H, N, d] = split_heads(x @ weight.T + bias) in one kernel.

    x: bf16 [B * N, d_model] (or [B, N, d_model]); weight: bf16 [3 H d, d_model];
    bias: bf16 [3 H d] or None."""
    import torch
    x2 = x.reshape(-1, x.shape[-1])
    for t in (x2, weight) + (() if bias is None else (bias,)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("qkv_projection: contiguous bf16 CUDA tensors")
    T, dm = x2.shape
    if T % batch:
        raise ValueError("qkv_projection: tokens not divisible by the batch size")
    N = T // batch
    shape = (batch, heads, N, head_dim)
    q, k, v = (torch.empty(shape, dtype=torch.bfloat16, device=x.device) if t is None else t
               for t in (q, k, v))
    code = library().fa_qkv_projection(_ptr(x2), _ptr(weight), _ptr(bias), _ptr(q), _ptr(k),
                                       _ptr(v), batch, N, heads, head_dim, dm,
                                       _stream_ptr(x.device))
    _check(code, "fa_qkv_projection")
    return q, k, v


from .paged_cache import PagedCache  # noqa: E402  (it uses the binding above)
