"""Thin ctypes binding of libgqa_paged.so (include/gqa_paged.h).

Argument marshalling only: torch tensors are checked for device, dtype, shape and
contiguity and passed as raw device pointers with the current CUDA stream; every step of
the computation runs in the library's kernels.  There is no fallback: if the library is
missing or the tensors are not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional, Tuple

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa_paged.so")

GQA_OK = 0
GQA_KV_BF16 = 0
GQA_KV_FP8_E4M3 = 1
GQA_KV_FP4 = 2
GQA_MAX_SPLITS = 64
GQA_SPLITS_BALANCED = -1

_lib = None
_fast = None
_fast_off = None  # why there is no compiled half
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_L = ctypes.c_int64

# name -> (restype, argtypes); the exported symbols of include/gqa_paged.h
SIGNATURES = {
    "gqa_paged_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "gqa_pick_splits": (_I, [_I, _I, _I, _I, _I]),
    "gqa_paged_decode": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                              ctypes.c_float, _I, _I, _P, _P, _P, _SZ, _P]),
    "gqa_paged_decode_partial": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                      ctypes.c_float, _I, _I, _P, _P, _P, _SZ, _P]),
    "gqa_paged_kt_build": (_I, [_P, _P, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "gqa_paged_kt_append": (_I, [_P, _P, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "gqa_paged_sparse_table_stride": (_I, [_I, _I, _I, _I]),
    "gqa_paged_sparse_select_workspace_size": (_SZ, [_I, _I, _I]),
    "gqa_paged_sparse_select": (_I, [_P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I,
                                     _P, _P, _P, _SZ, _P]),
    "gqa_paged_sparse_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "gqa_paged_sparse_decode": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                     ctypes.c_float, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "gqa_paged_decode_static_scratch": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I,
                                             _I, _I, _I, ctypes.c_float, _I, _I, _P, _P, _P]),
    "gqa_paged_prefill_workspace_size": (_SZ, [_I, _I, _I]),
    "gqa_paged_decode_kernel_launches": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "gqa_paged_prefill": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                               ctypes.c_float, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "lse_combine": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "gqa_paged_gather": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "gqa_paged_append_kv": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I,
                                 _P, _P]),
    "gqa_paged_write_kv": (_I, [_P, _P, _L, _L, _P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I,
                                _I, _I, _I, _I, _P, _P]),
    "gqa_paged_read_kv": (_I, [_P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _L,
                               _I, _P, _P, _P, _P]),
    "gqa_paged_append_decode": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _I,
                                     _I, _I, _I, ctypes.c_float, _I, _I, _P, _P, _P, _SZ, _P]),
    "gqa_get_error": (_I, [_P, _P]),
    "gqa_status_string": (ctypes.c_char_p, [_I]),
}


class GQAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


def load(path: Optional[str] = None):
    """Load the library (building it first if the sources are newer).  Raises when it
    cannot be built or loaded."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if path is None and (not os.path.exists(p) or _build._stale()):
        _build.build()
    if not os.path.exists(p):
        raise RuntimeError(f"libgqa_paged.so not found at {p}: the CUDA extension is required")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _load_fastcall(lib)
        _lib = lib
    return lib


def _load_fastcall(lib):
    """The compiled half of the hottest functions below (csrc/fastcall.cpp), on this library.  Where it
    cannot be built or loaded, their Python half makes every call."""
    global _fast, _fast_off
    _fast, _fast_off = None, _build.build_fastcall() if _build._fastcall_stale() else None
    if _fast_off is not None:
        return
    try:
        loader = importlib.machinery.ExtensionFileLoader("_fastcall", _build.FASTCALL)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fastcall", loader))
        loader.exec_module(module)
    except ImportError as e:
        _fast_off = str(e)
        return
    module.init(torch.Tensor,
                *(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
                    "gqa_paged_decode", "gqa_paged_decode_partial", "gqa_paged_append_kv",
                    "gqa_paged_append_decode", "gqa_paged_write_kv", "gqa_paged_read_kv")))
    _fast = module


def status_string(status: int) -> str:
    return load().gqa_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != GQA_OK:
        raise GQAError(fn, status)


# Plain ints, which ctypes converts by the signature: c_void_p and Stream objects cost 5 us a call.
def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _made(stream, make) -> torch.Tensor:
    """A buffer that a call makes for itself: of the stream that the call runs on, so that its zeros are
    there before the kernels and its memory is not reused before they are done."""
    if stream is None:
        return make()
    now = torch.cuda.current_stream()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    if stream.cuda_stream == now.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(now)  # (the caller may use and free it there)
    return t


def _empty(stream, shape, dtype, device) -> torch.Tensor:
    return _made(stream, lambda: torch.empty(shape, dtype=dtype, device=device))


def _scratch(stream, nbytes: int, device) -> torch.Tensor:
    return _made(stream, lambda: new_workspace(nbytes, device))


def _fast_call(fn: str, name: str, args, stream) -> bool:
    """Call `fn` of the compiled half: True if it was done.  False, with nothing done, for tensors
    that are not all as the function wants them: the caller's own checks then say what is wrong
    (or make the call, on tensors that only Python looks through)."""
    if _lib is None:
        load()
    if _fast is None:
        return False
    try:
        here = _get_device()
    except (RuntimeError, AssertionError):  # no GPU
        return False
    st = getattr(_fast, fn)(*args, here, None if stream is None else _stream(stream))
    if st is None:
        return False
    if st != GQA_OK:
        raise GQAError(name, st)
    return True


def _need(t: torch.Tensor, name: str, dtype=None, shape=None, here=None):
    """A contiguous CUDA tensor of this dtype and shape, on device `here` if one is given."""
    if (here is not None and isinstance(t, torch.Tensor) and t.get_device() == here
            and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype and \
            t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if here is not None and t.get_device() != here:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{here}")


def _device_of(k_pages: torch.Tensor) -> int:
    """The device of a call on these pools, which has to be the current one."""
    _need(k_pages, "k_pages", _KV_DTYPES)
    here = torch.cuda.current_device()
    if k_pages.get_device() != here:
        raise ValueError(f"k_pages is on cuda:{k_pages.get_device()}, the current device is cuda:{here}")
    return here


def _need_word(here: int, workspace: torch.Tensor):
    """A workspace with room for the error word."""
    _need(workspace, "workspace", torch.uint8, None, here)
    if workspace.numel() < 256:
        raise ValueError("workspace must have 256 bytes at least")


_KV_DTYPES = (torch.bfloat16, torch.uint8, torch.float8_e4m3fn)


# Bytes of a token's row in a 4-bit pool, 9 * head_dim / 16 -> head_dim.  No e4m3 pool has rows
# of these widths, so the last dimension tells the two uint8 pools apart.
_FP4_ROWS = {36: 64, 72: 128}


def _kv_layout(t: torch.Tensor) -> Tuple[int, int]:
    """(kv_dtype code, head_dim) of a pool [num_pages][Hk][P][row]."""
    if t.dim() != 4:
        raise ValueError("KV pools must be [num_pages][Hk][page_size][row]")
    row = t.shape[3]
    if t.dtype == torch.bfloat16:
        return GQA_KV_BF16, row
    if t.dtype == torch.uint8 and row in _FP4_ROWS:
        return GQA_KV_FP4, _FP4_ROWS[row]
    return GQA_KV_FP8_E4M3, row


def _need_scales(kv_dtype: int, num_pages: int, Hk: int, k_scale, v_scale, here=None):
    """e4m3 pools need scales [num_pages][Hk]; 4-bit pools take factors [Hk] or None."""
    if kv_dtype == GQA_KV_BF16:
        return
    if kv_dtype == GQA_KV_FP8_E4M3 and (k_scale is None or v_scale is None):
        raise ValueError("fp8 KV needs k_scale and v_scale")
    shape = (num_pages, Hk) if kv_dtype == GQA_KV_FP8_E4M3 else (Hk,)
    if k_scale is not None:
        _need(k_scale, "k_scale", torch.float32, shape, here)
    if v_scale is not None:
        _need(v_scale, "v_scale", torch.float32, shape, here)


def _four_bit_device(kv_dtype: int, k_pages: torch.Tensor) -> Optional[int]:
    """Calls on 4-bit pools take tensors of the current device alone; None for other pools."""
    return _device_of(k_pages) if kv_dtype == GQA_KV_FP4 else None


# ------------------------------------------------------------------------ raw ABI names

def gqa_pick_splits(B: int, Hk: int, max_seq_len: int, page_size: int, kv_dtype: int = 0) -> int:
    return load().gqa_pick_splits(B, Hk, max_seq_len, page_size, kv_dtype)


def gqa_paged_decode_workspace_size(B, Hq, Hk, head_dim, page_size, max_seq_len, kv_dtype,
                                    num_splits) -> int:
    return load().gqa_paged_decode_workspace_size(B, Hq, Hk, head_dim, page_size, max_seq_len,
                                                  kv_dtype, num_splits)


def gqa_paged_decode_kernel_launches(B, Hq, Hk, head_dim, page_size, max_seq_len, kv_dtype,
                                     num_splits, pack_gqa=True) -> int:
    return load().gqa_paged_decode_kernel_launches(B, Hq, Hk, head_dim, page_size, max_seq_len,
                                                   kv_dtype, num_splits, 1 if pack_gqa else 0)


def gqa_paged_prefill_workspace_size(total_q, Hq, head_dim) -> int:
    return load().gqa_paged_prefill_workspace_size(total_q, Hq, head_dim)


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled, 256-byte aligned workspace of at least nbytes.  One of them serves calls of
    every kind in turn on a stream, but for the balanced bf16 / e4m3 decode, which counts behind the
    header: give it one of its own, or zero it after a prefill, a sparse selection, a split decode or a
    balanced decode of fewer rows (include/gqa_paged.h)."""
    n = (max(int(nbytes), 256) + 255) // 256 * 256
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gqa_paged_decode(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                     page_table: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                     num_splits: int = 0, pack_gqa: bool = True,
                     k_scale: Optional[torch.Tensor] = None,
                     v_scale: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, want_lse: bool = True,
                     stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Paged GQA decode.  q bf16 [B][Hq][D]; pools [num_pages][Hk][P][D] bf16 or e4m3
    (uint8/float8_e4m3fn with fp32 scales [num_pages][Hk]), or 4-bit (new_fp4_pool; optional
    fp32 factors [Hk] as k_scale / v_scale); page_table int32 [B][pt_stride];
    seq_lens int32 [B].  Returns (out bf16 [B][Hq][D], lse fp32 [B][Hq] or None)."""
    if workspace is not None and out is not None and (lse is not None or not want_lse) and \
            _fast_call("decode", "gqa_paged_decode",
                       (False, q, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale, scale,
                        num_splits, pack_gqa, out, lse, workspace), stream):
        return out, lse
    _need(k_pages, "k_pages", _KV_DTYPES)
    kv_dtype, D2 = _kv_layout(k_pages)
    here = _four_bit_device(kv_dtype, k_pages)
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, here)
    _need(q, "q", torch.bfloat16, None, here)
    B, Hq, D = q.shape
    num_pages, Hk, P, _ = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and the KV pools differ")
    _need(page_table, "page_table", torch.int32, None, here)
    _need(seq_lens, "seq_lens", torch.int32, (B,), here)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pt_stride]")
    _need_scales(kv_dtype, num_pages, Hk, k_scale, v_scale, here)
    pt_stride = page_table.shape[1]
    if out is None:
        out = _empty(stream, (B, Hq, D), torch.bfloat16, q.device)
    _need(out, "out", torch.bfloat16, (B, Hq, D), here)
    if lse is None and want_lse:
        lse = _empty(stream, (B, Hq), torch.float32, q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq), here)
    if workspace is None:  # (a given one's size is checked by the call)
        workspace = _scratch(stream, gqa_paged_decode_workspace_size(
            B, Hq, Hk, D, P, pt_stride * P, kv_dtype, num_splits), q.device)
    _need(workspace, "workspace", torch.uint8, None, here)
    st = load().gqa_paged_decode(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), kv_dtype,
        _ptr(page_table), pt_stride, _ptr(seq_lens), B, Hq, Hk, D, P, num_pages, float(scale),
        int(num_splits), int(bool(pack_gqa)), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), _stream(stream))
    _check("gqa_paged_decode", st)
    return out, lse


def gqa_paged_decode_partial(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                             page_table: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                             num_splits: int = 0, pack_gqa: bool = True,
                             k_scale: Optional[torch.Tensor] = None,
                             v_scale: Optional[torch.Tensor] = None,
                             o_part: Optional[torch.Tensor] = None,
                             lse_part: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None,
                             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode over the tokens page_table / seq_lens cover, as one split's fp32 partial
    result: (o_part fp32 [B][Hq][D] normalised, lse_part fp32 [B][Hq]), the inputs
    lse_combine merges."""
    if workspace is not None and o_part is not None and lse_part is not None and \
            _fast_call("decode", "gqa_paged_decode_partial",
                       (True, q, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale, scale,
                        num_splits, pack_gqa, o_part, lse_part, workspace), stream):
        return o_part, lse_part
    _need(k_pages, "k_pages", _KV_DTYPES)
    kv_dtype, D2 = _kv_layout(k_pages)
    here = _four_bit_device(kv_dtype, k_pages)
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, here)
    _need(q, "q", torch.bfloat16, None, here)
    B, Hq, D = q.shape
    num_pages, Hk, P, _ = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and the KV pools differ")
    _need(page_table, "page_table", torch.int32, None, here)
    _need(seq_lens, "seq_lens", torch.int32, (B,), here)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pt_stride]")
    _need_scales(kv_dtype, num_pages, Hk, k_scale, v_scale, here)
    pt_stride = page_table.shape[1]
    if o_part is None:
        o_part = _empty(stream, (B, Hq, D), torch.float32, q.device)
    _need(o_part, "o_part", torch.float32, (B, Hq, D), here)
    if lse_part is None:
        lse_part = _empty(stream, (B, Hq), torch.float32, q.device)
    _need(lse_part, "lse_part", torch.float32, (B, Hq), here)
    if workspace is None:  # (a given one's size is checked by the call)
        workspace = _scratch(stream, gqa_paged_decode_workspace_size(
            B, Hq, Hk, D, P, pt_stride * P, kv_dtype, num_splits), q.device)
    _need(workspace, "workspace", torch.uint8, None, here)
    st = load().gqa_paged_decode_partial(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), kv_dtype,
        _ptr(page_table), pt_stride, _ptr(seq_lens), B, Hq, Hk, D, P, num_pages, float(scale),
        int(num_splits), int(bool(pack_gqa)), _ptr(o_part), _ptr(lse_part), _ptr(workspace),
        workspace.numel(), _stream(stream))
    _check("gqa_paged_decode_partial", st)
    return o_part, lse_part


def gqa_paged_decode_static_scratch(q: torch.Tensor, k_pages: torch.Tensor,
                                    v_pages: torch.Tensor, page_table: torch.Tensor,
                                    seq_lens: torch.Tensor, scale: float, num_splits: int = 0,
                                    pack_gqa: bool = True,
                                    k_scale: Optional[torch.Tensor] = None,
                                    v_scale: Optional[torch.Tensor] = None,
                                    out: Optional[torch.Tensor] = None,
                                    lse: Optional[torch.Tensor] = None,
                                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """gqa_paged_decode without a workspace: the library's fixed scratch array is used
    (for callers that cannot allocate device memory; see include/gqa_paged.h).  `out` and
    `lse` must be passed in by such callers; they are only created here for convenience."""
    _need(k_pages, "k_pages", _KV_DTYPES)
    kv_dtype, D2 = _kv_layout(k_pages)
    here = _four_bit_device(kv_dtype, k_pages)
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, here)
    _need(q, "q", torch.bfloat16, None, here)
    B, Hq, D = q.shape
    num_pages, Hk, P, _ = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and the KV pools differ")
    _need(page_table, "page_table", torch.int32, None, here)
    _need(seq_lens, "seq_lens", torch.int32, (B,), here)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pt_stride]")
    _need_scales(kv_dtype, num_pages, Hk, k_scale, v_scale, here)
    if out is None:
        out = _empty(stream, (B, Hq, D), torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(stream, (B, Hq), torch.float32, q.device)
    _need(out, "out", torch.bfloat16, (B, Hq, D), here)
    _need(lse, "lse", torch.float32, (B, Hq), here)
    st = load().gqa_paged_decode_static_scratch(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), kv_dtype,
        _ptr(page_table), page_table.shape[1], _ptr(seq_lens), B, Hq, Hk, D, P, num_pages,
        float(scale), int(num_splits), int(bool(pack_gqa)), _ptr(out), _ptr(lse),
        _stream(stream))
    _check("gqa_paged_decode_static_scratch", st)
    return out, lse


def _append_args(k_new, v_new, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale):
    _need(k_pages, "k_pages", _KV_DTYPES)
    kv_dtype, D = _kv_layout(k_pages)
    here = _four_bit_device(kv_dtype, k_pages)
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, here)
    num_pages, Hk, P, _ = k_pages.shape
    _need(seq_lens, "seq_lens", torch.int32, None, here)
    B = seq_lens.shape[0]
    _need(k_new, "k_new", torch.bfloat16, (B, Hk, D), here)
    _need(v_new, "v_new", torch.bfloat16, (B, Hk, D), here)
    _need(page_table, "page_table", torch.int32, None, here)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pt_stride]")
    _need_scales(kv_dtype, num_pages, Hk, k_scale, v_scale, here)
    return B, Hk, D, P, num_pages, kv_dtype, here


def gqa_paged_append_kv(k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor,
                        v_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                        k_scale: Optional[torch.Tensor] = None,
                        v_scale: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Write token seq_lens[b] - 1 of every sequence (k_new / v_new bf16 [B][Hk][D]) into
    the paged cache, in place (e4m3 and 4-bit pools quantise it; see include/gqa_paged.h).  Returns
    the workspace holding the error word."""
    if workspace is not None and _fast_call(
            "append_kv", "gqa_paged_append_kv",
            (k_new, v_new, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale, workspace),
            stream):
        return workspace
    B, Hk, D, P, num_pages, kv_dtype, here = _append_args(
        k_new, v_new, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale)
    if workspace is None:
        workspace = _scratch(stream, 256, k_pages.device)
    if kv_dtype == GQA_KV_FP4:
        _need_word(here, workspace)
    _need(workspace, "workspace", torch.uint8)
    st = load().gqa_paged_append_kv(
        _ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
        kv_dtype, _ptr(page_table), page_table.shape[1], _ptr(seq_lens), B, Hk, D, P, num_pages,
        _ptr(workspace), _stream(stream))
    _check("gqa_paged_append_kv", st)
    return workspace


def gqa_paged_append_decode(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                            k_pages: torch.Tensor, v_pages: torch.Tensor,
                            page_table: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                            num_splits: int = 0, pack_gqa: bool = True,
                            k_scale: Optional[torch.Tensor] = None,
                            v_scale: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, want_lse: bool = True,
                            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """gqa_paged_append_kv then gqa_paged_decode on one stream."""
    if workspace is not None and out is not None and (lse is not None or not want_lse) and \
            _fast_call("append_decode", "gqa_paged_append_decode",
                       (q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale,
                        scale, num_splits, pack_gqa, out, lse, workspace), stream):
        return out, lse
    B, Hk, D, P, num_pages, kv_dtype, here = _append_args(
        k_new, v_new, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale)
    _need(q, "q", torch.bfloat16, None, here)
    Bq, Hq, Dq = q.shape
    if Bq != B or Dq != D:
        raise ValueError("q must be [B][Hq][head_dim] with the pools' head_dim")
    pt_stride = page_table.shape[1]
    if out is None:
        out = _empty(stream, (B, Hq, D), torch.bfloat16, q.device)
    _need(out, "out", torch.bfloat16, (B, Hq, D), here)
    if lse is None and want_lse:
        lse = _empty(stream, (B, Hq), torch.float32, q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq), here)
    if workspace is None:  # (a given one's size is checked by the call)
        workspace = _scratch(stream, gqa_paged_decode_workspace_size(
            B, Hq, Hk, D, P, pt_stride * P, kv_dtype, num_splits), q.device)
    _need(workspace, "workspace", torch.uint8, None, here)
    st = load().gqa_paged_append_decode(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale),
        _ptr(v_scale), kv_dtype, _ptr(page_table), pt_stride, _ptr(seq_lens), B, Hq, Hk, D, P,
        num_pages, float(scale), int(num_splits), int(bool(pack_gqa)), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _check("gqa_paged_append_decode", st)
    return out, lse


def gqa_paged_prefill(q: torch.Tensor, cu_q: torch.Tensor, k_pages: torch.Tensor,
                      v_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                      scale: float, max_q_len: int, causal: bool = True,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, want_lse: bool = True,
                      stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal chunked prefill.  q bf16 [total_q][Hq][D]; cu_q int32 [B+1]; bf16 pools.  A workspace
    that a balanced bf16 / e4m3 decode uses too is zeroed in between (new_workspace)."""
    _need(q, "q", torch.bfloat16)
    T, Hq, D = q.shape
    _need(k_pages, "k_pages", torch.bfloat16)
    _need(v_pages, "v_pages", torch.bfloat16, k_pages.shape)
    num_pages, Hk, P, D2 = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and the KV pools differ")
    B = seq_lens.shape[0]
    _need(cu_q, "cu_q", torch.int32, (B + 1,))
    pt_stride = _table_on(None, page_table, B)
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = _empty(stream, (T, Hq, D), torch.bfloat16, q.device)
    _need(out, "out", torch.bfloat16, (T, Hq, D))
    if lse is None and want_lse:
        lse = _empty(stream, (T, Hq), torch.float32, q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, Hq))
    if workspace is None:
        workspace = _scratch(stream, gqa_paged_prefill_workspace_size(T, Hq, D), q.device)
    st = load().gqa_paged_prefill(
        _ptr(q), _ptr(cu_q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), pt_stride,
        _ptr(seq_lens), B, Hq, Hk, D, P, num_pages, float(scale), int(bool(causal)), T,
        int(max_q_len), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream))
    _check("gqa_paged_prefill", st)
    return out, lse


def lse_combine(o_part: torch.Tensor, lse_part: torch.Tensor,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Merge split results: o_part fp32 [S][rows][D], lse_part fp32 [S][rows]."""
    _need(o_part, "o_part", torch.float32)
    S, rows, D = o_part.shape
    _need(lse_part, "lse_part", torch.float32, (S, rows))
    if out is None:
        out = _empty(stream, (rows, D), torch.bfloat16, o_part.device)
    _need(out, "out", torch.bfloat16, (rows, D))
    if lse is None:
        lse = _empty(stream, rows, torch.float32, o_part.device)
    _need(lse, "lse", torch.float32, (rows,))
    st = load().lse_combine(_ptr(o_part), _ptr(lse_part), S, rows, D, _ptr(out), _ptr(lse),
                            _stream(stream))
    _check("lse_combine", st)
    return out, lse


def new_fp4_pool(num_pages: int, Hk: int, page_size: int, head_dim: int, device) -> torch.Tensor:
    """A zero-filled 4-bit pool of keys or of values: uint8 [num_pages][Hk][P][9 * D / 16]."""
    if head_dim not in (64, 128):
        raise ValueError("4-bit pools hold head_dim 64 or 128")
    return torch.zeros(num_pages, Hk, page_size, 9 * head_dim // 16, dtype=torch.uint8,
                       device=device)


def _need_rows(here: int, t: torch.Tensor, name: str, shape) -> int:
    """bf16 rows [T][Hk][D]: contiguous inside a row, any distance between rows, which is returned."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != here:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{here}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    T, Hk, D = shape
    if t.is_contiguous():
        return Hk * D
    if t.stride(2) != 1 or (Hk > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the [Hk][head_dim] values of a row must be contiguous")
    return t.stride(0) if T > 1 else Hk * D


def _pools_on(here: int, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale, v_scale):
    """Checks of the value pool and the scales; (kv_dtype, head_dim, num_pages, Hk, page_size)."""
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, here)
    kv_dtype, D = _kv_layout(k_pages)
    num_pages, Hk, P, _ = k_pages.shape
    _need_scales(kv_dtype, num_pages, Hk, k_scale, v_scale, here)
    return kv_dtype, D, num_pages, Hk, P


def _table_on(here: Optional[int], page_table: torch.Tensor, B: int) -> int:
    _need(page_table, "page_table", torch.int32, None, here)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pt_stride]")
    return page_table.shape[1]


def gqa_paged_write_kv(k_new: torch.Tensor, v_new: torch.Tensor, cu_q: torch.Tensor,
                       k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, max_q_len: int,
                       k_scale: Optional[torch.Tensor] = None,
                       v_scale: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Write the newest cu_q[b+1] - cu_q[b] tokens of every sequence (k_new / v_new bf16
    [total_q][Hk][D], rows of any stride; cu_q int32 [B+1]) into the paged cache, in place;
    e4m3 and 4-bit pools quantise them (see include/gqa_paged.h).  Returns the workspace holding
    the error word."""
    if workspace is not None and _fast_call(
            "write_kv", "gqa_paged_write_kv",
            (k_new, v_new, cu_q, k_pages, v_pages, page_table, seq_lens, k_scale, v_scale,
             max_q_len, workspace), stream):
        return workspace
    here = _device_of(k_pages)
    kv_dtype, D, num_pages, Hk, P = _pools_on(here, k_pages, v_pages, k_scale, v_scale)
    _need(seq_lens, "seq_lens", torch.int32, None, here)
    B, T = seq_lens.shape[0], k_new.shape[0]
    ks = _need_rows(here, k_new, "k_new", (T, Hk, D))
    vs = _need_rows(here, v_new, "v_new", (T, Hk, D))
    _need(cu_q, "cu_q", torch.int32, (B + 1,), here)
    pt_stride = _table_on(here, page_table, B)
    if workspace is None:
        workspace = _scratch(stream, 256, k_pages.device)
    _need_word(here, workspace)
    if T == 0:
        return workspace
    st = load().gqa_paged_write_kv(
        _ptr(k_new), _ptr(v_new), ks, vs, _ptr(cu_q), _ptr(k_pages), _ptr(v_pages),
        _ptr(k_scale), _ptr(v_scale), kv_dtype, _ptr(page_table), pt_stride,
        _ptr(seq_lens), B, Hk, D, P, num_pages, T, int(max_q_len), _ptr(workspace),
        _stream(stream))
    _check("gqa_paged_write_kv", st)
    return workspace


def gqa_paged_read_kv(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                      seq_lens: torch.Tensor, cu_out: torch.Tensor, total: int,
                      starts: Optional[torch.Tensor] = None,
                      k_scale: Optional[torch.Tensor] = None,
                      v_scale: Optional[torch.Tensor] = None, paged: bool = False,
                      k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Tokens starts[b] (default 0) .. seq_lens[b] - 1 of every sequence as bf16 values, from
    bf16, e4m3 or 4-bit pools: (k, v) [total][Hk][D] rows at cu_out (int64 [B+1]), or, with
    `paged`, bf16 pages [total][Hk][P][D] with cu_out counting pages (page cu_out[b] + i holds
    the i-th page of the stretch; slots outside it are not written)."""
    if workspace is not None and k_out is not None and v_out is not None and _fast_call(
            "read_kv", "gqa_paged_read_kv",
            (k_pages, v_pages, page_table, seq_lens, k_scale, v_scale, starts, cu_out, total,
             paged, k_out, v_out, workspace), stream):
        return k_out, v_out
    here = _device_of(k_pages)
    kv_dtype, D, num_pages, Hk, P = _pools_on(here, k_pages, v_pages, k_scale, v_scale)
    _need(seq_lens, "seq_lens", torch.int32, None, here)
    B = seq_lens.shape[0]
    pt_stride = _table_on(here, page_table, B)
    _need(cu_out, "cu_out", torch.int64, (B + 1,), here)
    if starts is not None:
        _need(starts, "starts", torch.int32, (B,), here)
    total = int(total)
    shape = (total, Hk, P, D) if paged else (total, Hk, D)
    if k_out is None:
        k_out = _empty(stream, shape, torch.bfloat16, k_pages.device)
    if v_out is None:
        v_out = _empty(stream, shape, torch.bfloat16, k_pages.device)
    _need(k_out, "k_out", torch.bfloat16, shape, here)
    _need(v_out, "v_out", torch.bfloat16, shape, here)
    if workspace is None:
        workspace = _scratch(stream, 256, k_pages.device)
    _need_word(here, workspace)
    if total == 0:
        return k_out, v_out
    st = load().gqa_paged_read_kv(
        _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), kv_dtype, _ptr(page_table),
        pt_stride, _ptr(starts), _ptr(seq_lens), _ptr(cu_out), B, Hk, D, P, num_pages,
        total, int(bool(paged)), _ptr(k_out), _ptr(v_out), _ptr(workspace), _stream(stream))
    _check("gqa_paged_read_kv", st)
    return k_out, v_out


def gqa_paged_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                     seq_lens: torch.Tensor, cu_kv: torch.Tensor, total: int,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Bit-exact copy-out of the paged cache: returns (k, v) [total][Hk][D]."""
    _need(k_pages, "k_pages", _KV_DTYPES)
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape)
    num_pages, Hk, P, D = k_pages.shape
    B = seq_lens.shape[0]
    pt_stride = _table_on(None, page_table, B)
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _need(cu_kv, "cu_kv", torch.int64, (B + 1,))
    ko = _empty(stream, (total, Hk, D), k_pages.dtype, k_pages.device)
    vo = _empty(stream, (total, Hk, D), k_pages.dtype, k_pages.device)
    st = load().gqa_paged_gather(_ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                 pt_stride, _ptr(seq_lens), _ptr(cu_kv), B, Hk, D, P,
                                 num_pages, k_pages.element_size(), _ptr(ko), _ptr(vo),
                                 _stream(stream))
    _check("gqa_paged_gather", st)
    return ko, vo


def gqa_get_error(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream, return and clear the device error word of `workspace`."""
    _need(workspace, "workspace", torch.uint8)
    return load().gqa_get_error(_ptr(workspace), _stream(stream))


# ------------------------------------------------------------------------ sparse decode

def _sparse_common(q, k_pages, page_table, seq_lens):
    _need(q, "q", torch.bfloat16)
    B, Hq, D = q.shape
    _need(k_pages, "k_pages", torch.bfloat16)
    num_pages, Hk, P, D2 = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and the KV pools differ")
    _need(page_table, "page_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B][pt_stride]")
    return B, Hq, Hk, D, P, num_pages, page_table.shape[1]


def new_kt_cache(k_pages: torch.Tensor) -> torch.Tensor:
    """An empty KT cache for a bf16 pool: bf16 [num_pages][Hk][D][2]."""
    num_pages, Hk, P, D = k_pages.shape
    return torch.zeros(num_pages, Hk, D, 2, dtype=torch.bfloat16, device=k_pages.device)


def gqa_paged_kt_build(k_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                       kt: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """KT entries (per page and kv head: min and max of the keys over the valid tokens)
    of every page the sequences reference; returns kt bf16 [num_pages][Hk][D][2]."""
    _need(k_pages, "k_pages", torch.bfloat16)
    num_pages, Hk, P, D = k_pages.shape
    _need(seq_lens, "seq_lens", torch.int32)
    B = seq_lens.shape[0]
    pt_stride = _table_on(None, page_table, B)
    if kt is None:
        kt = _made(stream, lambda: new_kt_cache(k_pages))
    _need(kt, "kt", torch.bfloat16, (num_pages, Hk, D, 2))
    if workspace is None:
        workspace = _scratch(stream, 256, k_pages.device)
    st = load().gqa_paged_kt_build(_ptr(k_pages), _ptr(page_table), pt_stride,
                                   _ptr(seq_lens), B, Hk, D, P, num_pages, _ptr(kt),
                                   _ptr(workspace), _stream(stream))
    _check("gqa_paged_kt_build", st)
    return kt


def gqa_paged_kt_append(k_new: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                        kt: torch.Tensor, page_size: int,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Update the KT entries with the token at position seq_lens[b] - 1 (k_new bf16
    [B][Hk][D]), in place."""
    _need(k_new, "k_new", torch.bfloat16)
    B, Hk, D = k_new.shape
    num_pages = kt.shape[0]
    _need(kt, "kt", torch.bfloat16, (num_pages, Hk, D, 2))
    pt_stride = _table_on(None, page_table, B)
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if workspace is None:
        workspace = _scratch(stream, 256, kt.device)
    st = load().gqa_paged_kt_append(_ptr(k_new), _ptr(page_table), pt_stride,
                                    _ptr(seq_lens), B, Hk, D, int(page_size), num_pages, _ptr(kt),
                                    _ptr(workspace), _stream(stream))
    _check("gqa_paged_kt_append", st)
    return kt


def gqa_paged_sparse_table_stride(pt_stride: int, page_size: int, topk: int, window: int) -> int:
    return load().gqa_paged_sparse_table_stride(pt_stride, page_size, topk, window)


def gqa_paged_sparse_select(q: torch.Tensor, kt: torch.Tensor, k_pages: torch.Tensor,
                            page_table: torch.Tensor, seq_lens: torch.Tensor, topk: int,
                            window: int, workspace: Optional[torch.Tensor] = None,
                            stream=None):
    """The chosen pages: returns (sel_table int32 [B*Hk][ss] of physical*Hk + kv head,
    sel_lens int32 [B*Hk], sel_pages int32 [B*Hk][ss] logical pages).  A workspace that a balanced
    bf16 / e4m3 decode uses too is zeroed in between (new_workspace)."""
    B, Hq, Hk, D, P, num_pages, pts = _sparse_common(q, k_pages, page_table, seq_lens)
    _need(kt, "kt", torch.bfloat16, (num_pages, Hk, D, 2))
    ss = gqa_paged_sparse_table_stride(pts, P, topk, window)
    dev = q.device
    sel_table = _made(stream, lambda: torch.full((B * Hk, max(ss, 1)), -1, dtype=torch.int32, device=dev))
    sel_pages = _made(stream, lambda: torch.full((B * Hk, max(ss, 1)), -1, dtype=torch.int32, device=dev))
    sel_lens = _made(stream, lambda: torch.zeros(B * Hk, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = _scratch(stream, load().gqa_paged_sparse_select_workspace_size(B, Hk, pts), dev)
    st = load().gqa_paged_sparse_select(_ptr(q), _ptr(kt), _ptr(page_table), pts, _ptr(seq_lens),
                                        B, Hq, Hk, D, P, num_pages, int(topk), int(window),
                                        _ptr(sel_table), max(ss, 1), _ptr(sel_lens),
                                        _ptr(sel_pages), _ptr(workspace), workspace.numel(),
                                        _stream(stream))
    _check("gqa_paged_sparse_select", st)
    return sel_table, sel_lens, sel_pages


def gqa_paged_sparse_decode_workspace_size(B, Hq, Hk, head_dim, page_size, pt_stride, topk,
                                           window, num_splits=0) -> int:
    return load().gqa_paged_sparse_decode_workspace_size(B, Hq, Hk, head_dim, page_size,
                                                         pt_stride, topk, window, num_splits)


def gqa_paged_sparse_decode(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                            kt: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                            scale: float, topk: int, window: int, num_splits: int = 0,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, want_lse: bool = True,
                            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Page-level top-K sparse decode (bf16 pools): the window pages plus the topk
    best-scoring earlier pages of every (sequence, kv head) are attended.  The workspace holds a
    balanced decode's counters (new_workspace)."""
    B, Hq, Hk, D, P, num_pages, pts = _sparse_common(q, k_pages, page_table, seq_lens)
    _need(v_pages, "v_pages", torch.bfloat16, k_pages.shape)
    _need(kt, "kt", torch.bfloat16, (num_pages, Hk, D, 2))
    if out is None:
        out = _empty(stream, (B, Hq, D), torch.bfloat16, q.device)
    _need(out, "out", torch.bfloat16, (B, Hq, D))
    if lse is None and want_lse:
        lse = _empty(stream, (B, Hq), torch.float32, q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq))
    need = gqa_paged_sparse_decode_workspace_size(B, Hq, Hk, D, P, pts, topk, window, num_splits)
    if workspace is None:
        workspace = _scratch(stream, need, q.device)
    _need(workspace, "workspace", torch.uint8)
    st = load().gqa_paged_sparse_decode(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kt), _ptr(page_table), pts, _ptr(seq_lens),
        B, Hq, Hk, D, P, num_pages, float(scale), int(topk), int(window), int(num_splits),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("gqa_paged_sparse_decode", st)
    return out, lse
