"""ctypes binding of the C ABI declared in include/attn_gb300.h.

Argument marshalling only: shapes are read off the torch tensors, pointers and
the current CUDA stream are handed to the library, and a non-zero status
raises ``AttnError``.  Every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the shared library has not been built
(``__graft_entry__.build()`` or ``python -m attn_fwd_02_gb300.build``), every
call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libattn_gb300.so"
_lib = None
_lock = threading.Lock()

ATTN_OK = 0
_STATUS_NAMES = {
    0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_MISALIGNED",
    4: "ATTN_ERR_WORKSPACE", 5: "ATTN_ERR_CUDA", 6: "ATTN_ERR_DEVICE_TIMEOUT", 7: "ATTN_ERR_SCRATCH_LIMIT",
}

# name -> (restype, argtypes); mirrors include/attn_gb300.h
P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "attn_fwd": (I, [P, P, P, P, P, I, I, I, I, I, I, F, P]),
    "attn_fwd_kvlen": (I, [P, P, P, P, P, I, I, I, I, I, I, F, P, P]),
    "attn_fwd_gqa": (I, [P, P, P, P, P, I, I, I, I, I, I, I, F, P, P]),
    "paged_attn_decode_workspace_size": (Z, [I, I, I, I, I]),
    "paged_attn_decode_workspace_size_ctx": (Z, [I, I, I, I]),
    "paged_attn_decode_gqa_workspace_size": (Z, [I, I, I, I, I, I]),
    "paged_attn_decode": (I, [P, P, P, P, P, I, P, P, I, I, I, I, I, F, P, Z, P]),
    "paged_attn_decode_noalloc": (I, [P, P, P, P, P, I, P, P, I, I, I, I, I, F, P]),
    "paged_attn_decode_gqa": (I, [P, P, P, P, P, I, P, P, I, I, I, I, I, I, F, P, Z, P]),
    "paged_attn_prefill": (I, [P, P, P, P, P, I, P, P, I, I, I, I, I, I, I, I, F, P]),
    "paged_kv_append": (I, [P, P, P, P, P, P, I, I, I, I, I, I, I, P]),
    "attn_bwd_workspace_size": (Z, [I, I, I]),
    "paged_attn_decode_fp8": (I, [P, P, P, F, F, P, P, I, P, P, I, I, I, I, I, I, F, P, Z, P]),
    "kv_quantize_fp8": (I, [P, P, Z, F, P]),
    "paged_attn_prefill_fp8": (I, [P, P, P, F, F, P, P, I, P, P, I, I, I, I, I, I, I, I, F, P]),
    "paged_kv_append_fp8": (I, [P, P, P, P, F, F, P, P, I, I, I, I, I, I, I, P]),
    "attn_bwd": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, Z, P]),
    "paged_kv_append_rope": (I, [P, P, P, P, P, P, P, P, P, P, I, I, I, P, P, P, I, I, I, I, I, I, I, I, P]),
    "paged_kv_append_rope_fp8": (I, [P, P, P, P, P, P, P, P, P, F, F, P, I, I, I, P, P, P, I, I, I, I, I, I, I, I, P]),
    "attn_fwd_scoremod": (I, [P, P, P, P, P, I, I, I, I, I, I, I, F, F, P, P, P, P, P]),
    "attn_bwd_scoremod_workspace_size": (Z, [I, I, I, I, I, I]),
    "attn_bwd_scoremod": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, F, P, P, P, P, P, Z, P]),
    "paged_attn_decode_scoremod_workspace_size": (Z, [I, I, I, I, I, I]),
    "paged_attn_decode_scoremod": (I, [P, P, P, P, P, I, P, P, I, I, I, I, I, I, F, F, P, P, P, Z, P]),
    "paged_attn_decode_scoremod_fp8": (I, [P, P, P, F, F, P, P, I, P, P, I, I, I, I, I, I, F, F, P, P, P, Z, P]),
    "paged_attn_decode_shared_workspace_size": (Z, [I, I, I, I, I, I, I]),
    "paged_attn_decode_shared": (I, [P, P, P, P, P, P, I, I, P, P, I, I, I, I, I, I, F, P, Z, P]),
    "paged_attn_decode_shared_fp8": (I, [P, P, P, F, F, P, P, P, I, I, P, P, I, I, I, I, I, I, F, P, Z, P]),
    "attn_check_device_status": (I, [P]),
    "attn_last_device_status": (I, []),
    "attn_selftest_bounded_wait": (I, [P]),
    "attn_status_string": (ctypes.c_char_p, [I]),
    "attn_version": (ctypes.c_char_p, []),
}


class AttnError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed: {_STATUS_NAMES.get(status, status)} ({text})")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, LIB_NAME)


def load_library():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{LIB_NAME} is not built; run `python -m attn_fwd_02_gb300.build` "
                    "(there is no CPU fallback)")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def attn_status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != ATTN_OK:
        raise AttnError(fn, status, attn_status_string(status))


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, name, dtype, ndim):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out_like(out, like, name):
    """``out`` given by the caller must match ``like`` (dtype, shape, device) and be contiguous;
    None allocates one with torch."""
    import torch
    if out is None:
        return torch.empty_like(like)
    _require(out, name, like.dtype, like.dim())
    if tuple(out.shape) != tuple(like.shape) or out.device != like.device:
        raise ValueError(f"{name} must be {tuple(like.shape)} on {like.device}, got {tuple(out.shape)} "
                         f"on {out.device}")
    return out


def _lse_out(lse, shape, device, want: bool):
    """fp32 log-sum-exp output of the given shape on ``device``: checked if given, allocated
    if None and wanted."""
    import torch
    if lse is None:
        return torch.empty(shape, dtype=torch.float32, device=device) if want else None
    _require(lse, "lse", torch.float32, len(shape))
    if tuple(lse.shape) != tuple(shape) or lse.device != device:
        raise ValueError(f"lse must be {tuple(shape)} on {device}, got {tuple(lse.shape)} on {lse.device}")
    return lse


def attn_fwd_kvlen(q, k, v, causal: bool, scale: float | None = None, kv_lens=None,
                   out=None, lse=None, return_lse: bool = True, stream=None):
    """Prefill attention. q [B,H,Nq,d], k/v [B,H,Nkv,d] bf16 CUDA tensors;
    kv_lens optional int32 [B] CUDA tensor.  Returns (o, lse)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16, 4)
    B, H, Nq, d = q.shape
    Nkv = k.shape[2]
    if tuple(k.shape) != (B, H, Nkv, d) or tuple(v.shape) != (B, H, Nkv, d):
        raise ValueError("k and v must be [B, H, Nkv, d] matching q")
    if kv_lens is not None:
        _require(kv_lens, "kv_lens", torch.int32, 1)
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H, Nq), q.device, return_lse)
    lib = load_library()
    st = lib.attn_fwd_kvlen(_dptr(q), _dptr(k), _dptr(v), _dptr(out), _dptr(lse), B, H, Nq, Nkv, d,
                            int(bool(causal)), float(scale), _dptr(kv_lens), _stream_ptr(stream))
    _check("attn_fwd_kvlen", st)
    return out, lse


def attn_fwd_gqa(q, k, v, causal: bool, scale: float | None = None, kv_lens=None, out=None, lse=None,
                 return_lse: bool = True, stream=None):
    """Grouped-query prefill: q [B,Hq,Nq,d], k/v [B,Hkv,Nkv,d] bf16 CUDA tensors with
    Hq % Hkv == 0 (query head h reads key/value head h // (Hq // Hkv)).  Returns (o, lse)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16, 4)
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Nkv, d) or tuple(v.shape) != (B, Hkv, Nkv, d):
        raise ValueError("k and v must be [B, Hkv, Nkv, d] matching q")
    if kv_lens is not None:
        _require(kv_lens, "kv_lens", torch.int32, 1)
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, Hq, Nq), q.device, return_lse)
    st = load_library().attn_fwd_gqa(_dptr(q), _dptr(k), _dptr(v), _dptr(out), _dptr(lse), B, Hq, Hkv, Nq, Nkv,
                                     d, int(bool(causal)), float(scale), _dptr(kv_lens), _stream_ptr(stream))
    _check("attn_fwd_gqa", st)
    return out, lse


def kv_quantize_fp8(x, scale: float, out=None, stream=None):
    """bf16 CUDA tensor -> uint8 e4m3 codes of the same shape under a per-tensor scale
    (value = e4m3(code) * scale; code = nearest-even e4m3 of fp32(x) * fp32(1/scale), saturating)."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous bf16 CUDA tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    else:
        _require(out, "out", torch.uint8, x.dim())
        if tuple(out.shape) != tuple(x.shape) or out.device != x.device:
            raise ValueError("out must be a uint8 tensor of x's shape on x's device")
    st = load_library().kv_quantize_fp8(_dptr(x), _dptr(out), x.numel(), float(scale), _stream_ptr(stream))
    _check("kv_quantize_fp8", st)
    return out


def paged_kv_append_fp8(k_new, v_new, k_pages, v_pages, k_scale: float, v_scale: float, page_table, start_pos,
                        stream=None):
    """paged_kv_append into an e4m3 cache (k_pages/v_pages uint8 [P,Hkv,16,d]); new K/V bf16
    [B,Hkv,Nnew,d] are converted with the cache's scales."""
    import torch
    _require(k_new, "k_new", torch.bfloat16, 4)
    _require(v_new, "v_new", torch.bfloat16, 4)
    _require(k_pages, "k_pages", torch.uint8, 4)
    _require(v_pages, "v_pages", torch.uint8, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(start_pos, "start_pos", torch.int32, 1)
    B, Hkv, Nnew, d = k_new.shape
    P, Hk, ps, dk = k_pages.shape
    if (Hk, dk) != (Hkv, d) or tuple(v_new.shape) != tuple(k_new.shape) or tuple(v_pages.shape) != tuple(
            k_pages.shape):
        raise ValueError("shape mismatch between new K/V and the pages")
    st = load_library().paged_kv_append_fp8(_dptr(k_new), _dptr(v_new), _dptr(k_pages), _dptr(v_pages),
                                            float(k_scale), float(v_scale), _dptr(page_table), _dptr(start_pos), ps,
                                            B, Hkv, Nnew, d, page_table.shape[1], P, _stream_ptr(stream))
    _check("paged_kv_append_fp8", st)


def paged_attn_decode_fp8(q, k_pages, v_pages, k_scale: float, v_scale: float, page_table, ctx_lens,
                          scale: float | None = None, out=None, lse=None, workspace=None, return_lse: bool = True,
                          stream=None):
    """Paged decode over an e4m3 cache: q [B,H,d] bf16; k_pages/v_pages uint8 codes [P,Hkv,16,d]
    with per-tensor scales.  Returns (o, lse)."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_pages, "k_pages", torch.uint8, 4)
    _require(v_pages, "v_pages", torch.uint8, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(ctx_lens, "ctx_lens", torch.int32, 1)
    B, H, d = q.shape
    P, Hkv, ps, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, d]")
    if scale is None:
        scale = d ** -0.5
    max_pages = page_table.shape[1]
    lib = load_library()
    need = int(lib.paged_attn_decode_gqa_workspace_size(B, H, Hkv, d, max_pages, ps))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H), q.device, return_lse)
    st = lib.paged_attn_decode_fp8(_dptr(q), _dptr(k_pages), _dptr(v_pages), float(k_scale), float(v_scale),
                                   _dptr(page_table), _dptr(ctx_lens), ps, _dptr(out), _dptr(lse), B, H, Hkv, d,
                                   max_pages, P, float(scale), _dptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check("paged_attn_decode_fp8", st)
    return out, lse


def attn_bwd_workspace_size(B: int, Hq: int, Nq: int) -> int:
    return int(load_library().attn_bwd_workspace_size(B, Hq, Nq))


def attn_bwd(q, k, v, o, lse, dout, causal: bool, scale: float | None = None, kv_lens=None,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of attn_fwd_gqa: q, o, dout [B,Hq,Nq,d] and k, v [B,Hkv,Nkv,d] bf16 CUDA tensors,
    lse [B,Hq,Nq] fp32 from the forward; causal, scale and kv_lens as in the forward call.
    Returns (dq, dk, dv) bf16.  The workspace (uint8, attn_bwd_workspace_size bytes) ends up
    holding the row term D [B,Hq,Nq] fp32."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _require(t, n, torch.bfloat16, 4)
    _require(lse, "lse", torch.float32, 3)
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Nkv, d) or tuple(v.shape) != (B, Hkv, Nkv, d):
        raise ValueError("k and v must be [B, Hkv, Nkv, d] matching q")
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("o and dout must match q, lse must be [B, Hq, Nq]")
    if kv_lens is not None:
        _require(kv_lens, "kv_lens", torch.int32, 1)
    if scale is None:
        scale = d ** -0.5
    dq = _out_like(dq, q, "dq")
    dk = _out_like(dk, k, "dk")
    dv = _out_like(dv, v, "dv")
    lib = load_library()
    need = int(lib.attn_bwd_workspace_size(B, Hq, Nq))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib.attn_bwd(_dptr(q), _dptr(k), _dptr(v), _dptr(o), _dptr(lse), _dptr(dout), _dptr(dq), _dptr(dk),
                      _dptr(dv), B, Hq, Hkv, Nq, Nkv, d, int(bool(causal)), float(scale), _dptr(kv_lens),
                      _dptr(workspace), workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check("attn_bwd", st)
    return dq, dk, dv


def attn_fwd(q, k, v, causal: bool, scale: float | None = None, out=None, lse=None,
             return_lse: bool = True, stream=None):
    """Prefill attention without key padding (calls the C entry point attn_fwd)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16, 4)
    B, H, Nq, d = q.shape
    Nkv = k.shape[2]
    if tuple(k.shape) != (B, H, Nkv, d) or tuple(v.shape) != (B, H, Nkv, d):
        raise ValueError("k and v must be [B, H, Nkv, d] matching q")
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H, Nq), q.device, return_lse)
    lib = load_library()
    st = lib.attn_fwd(_dptr(q), _dptr(k), _dptr(v), _dptr(out), _dptr(lse), B, H, Nq, Nkv, d,
                      int(bool(causal)), float(scale), _stream_ptr(stream))
    _check("attn_fwd", st)
    return out, lse


def paged_attn_decode_workspace_size(B: int, H: int, d: int, max_pages_per_seq: int,
                                     page_size: int = 16) -> int:
    return int(load_library().paged_attn_decode_workspace_size(B, H, d, max_pages_per_seq, page_size))


def paged_attn_decode_workspace_size_ctx(B: int, H: int, d: int, max_ctx_len: int) -> int:
    return int(load_library().paged_attn_decode_workspace_size_ctx(B, H, d, max_ctx_len))


def paged_attn_decode_gqa_workspace_size(B: int, H: int, Hkv: int, d: int, max_pages_per_seq: int,
                                         page_size: int = 16) -> int:
    return int(load_library().paged_attn_decode_gqa_workspace_size(B, H, Hkv, d, max_pages_per_seq, page_size))


def paged_attn_decode(q, k_pages, v_pages, page_table, ctx_lens, scale: float | None = None,
                      out=None, lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Paged decode. q [B,H,d]; k_pages/v_pages [P,H,page_size,d] bf16; page_table
    [B,max_pages] int32; ctx_lens [B] int32 (all CUDA).  ``workspace``: optional uint8
    CUDA tensor of at least paged_attn_decode_workspace_size() bytes (allocated with torch
    here if not given).  Returns (o, lse)."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_pages, "k_pages", torch.bfloat16, 4)
    _require(v_pages, "v_pages", torch.bfloat16, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(ctx_lens, "ctx_lens", torch.int32, 1)
    B, H, d = q.shape
    num_pages, Hk, page_size, dk = k_pages.shape
    if (Hk, dk) != (H, d) or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages must be [num_pages, H, page_size, d] matching q")
    if page_table.shape[0] != B or ctx_lens.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and ctx_lens [B]")
    max_pages = page_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H), q.device, return_lse)
    lib = load_library()
    need = int(lib.paged_attn_decode_workspace_size(B, H, d, max_pages, page_size))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib.paged_attn_decode(_dptr(q), _dptr(k_pages), _dptr(v_pages), _dptr(page_table),
                               _dptr(ctx_lens), page_size, _dptr(out), _dptr(lse), B, H, d,
                               max_pages, num_pages, float(scale), _dptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check("paged_attn_decode", st)
    return out, lse


def paged_attn_decode_gqa(q, k_pages, v_pages, page_table, ctx_lens, scale: float | None = None,
                          out=None, lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Grouped-query paged decode: q [B,H,d]; k_pages/v_pages [P,Hkv,page_size,d] with
    H % Hkv == 0; page_table [B,max_pages] int32; ctx_lens [B] int32.  Returns (o, lse)."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_pages, "k_pages", torch.bfloat16, 4)
    _require(v_pages, "v_pages", torch.bfloat16, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(ctx_lens, "ctx_lens", torch.int32, 1)
    B, H, d = q.shape
    num_pages, Hkv, page_size, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d] matching q")
    if page_table.shape[0] != B or ctx_lens.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and ctx_lens [B]")
    max_pages = page_table.shape[1]
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H), q.device, return_lse)
    lib = load_library()
    need = int(lib.paged_attn_decode_gqa_workspace_size(B, H, Hkv, d, max_pages, page_size))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = lib.paged_attn_decode_gqa(_dptr(q), _dptr(k_pages), _dptr(v_pages), _dptr(page_table), _dptr(ctx_lens),
                                   page_size, _dptr(out), _dptr(lse), B, H, Hkv, d, max_pages, num_pages,
                                   float(scale), _dptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream_ptr(stream))
    _check("paged_attn_decode_gqa", st)
    return out, lse


def paged_attn_decode_noalloc(q, k_pages, v_pages, page_table, ctx_lens, scale: float | None = None,
                              out=None, lse=None, return_lse: bool = True, stream=None):
    """paged_attn_decode without a workspace, for callers that cannot allocate device
    memory: the library keeps the chunk partials in its own fixed 12 MiB device array.
    Pass ``out`` (bf16, q's shape) and ``lse`` (fp32 [B, H]), both contiguous on q's device,
    to avoid any allocation here as well.  Calls that may overlap on the GPU share that
    array and must be ordered by the caller.
    Returns (o, lse)."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_pages, "k_pages", torch.bfloat16, 4)
    _require(v_pages, "v_pages", torch.bfloat16, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(ctx_lens, "ctx_lens", torch.int32, 1)
    B, H, d = q.shape
    num_pages, Hk, page_size, dk = k_pages.shape
    if (Hk, dk) != (H, d) or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages must be [num_pages, H, page_size, d] matching q")
    if page_table.shape[0] != B or ctx_lens.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and ctx_lens [B]")
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H), q.device, return_lse)
    st = load_library().paged_attn_decode_noalloc(
        _dptr(q), _dptr(k_pages), _dptr(v_pages), _dptr(page_table), _dptr(ctx_lens), page_size, _dptr(out),
        _dptr(lse), B, H, d, page_table.shape[1], num_pages, float(scale), _stream_ptr(stream))
    _check("paged_attn_decode_noalloc", st)
    return out, lse


def paged_attn_prefill(q, k_pages, v_pages, page_table, ctx_lens, causal: bool, scale: float | None = None,
                       out=None, lse=None, return_lse: bool = True, stream=None):
    """Chunked prefill over the paged cache: q [B,H,Nq,d] are the last Nq of the ctx_lens[b]
    cached tokens of each sequence; k_pages/v_pages [P,Hkv,page_size,d]; page_table
    [B,max_pages] int32; ctx_lens [B] int32 (all CUDA).  Returns (o, lse)."""
    import torch
    _require(q, "q", torch.bfloat16, 4)
    _require(k_pages, "k_pages", torch.bfloat16, 4)
    _require(v_pages, "v_pages", torch.bfloat16, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(ctx_lens, "ctx_lens", torch.int32, 1)
    B, H, Nq, d = q.shape
    num_pages, Hkv, page_size, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d] matching q")
    if page_table.shape[0] != B or ctx_lens.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and ctx_lens [B]")
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H, Nq), q.device, return_lse)
    st = load_library().paged_attn_prefill(_dptr(q), _dptr(k_pages), _dptr(v_pages), _dptr(page_table),
                                           _dptr(ctx_lens), page_size, _dptr(out), _dptr(lse), B, H, Hkv, Nq, d,
                                           page_table.shape[1], num_pages, int(bool(causal)), float(scale),
                                           _stream_ptr(stream))
    _check("paged_attn_prefill", st)
    return out, lse


def paged_attn_prefill_fp8(q, k_pages, v_pages, k_scale: float, v_scale: float, page_table, ctx_lens,
                           causal: bool, scale: float | None = None, out=None, lse=None, return_lse: bool = True,
                           stream=None):
    """paged_attn_prefill over an e4m3 cache: q [B,H,Nq,d] bf16; k_pages/v_pages uint8 codes
    [P,Hkv,16,d] with per-tensor scales (value = e4m3(code) * scale).  Returns (o, lse)."""
    import torch
    _require(q, "q", torch.bfloat16, 4)
    _require(k_pages, "k_pages", torch.uint8, 4)
    _require(v_pages, "v_pages", torch.uint8, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(ctx_lens, "ctx_lens", torch.int32, 1)
    B, H, Nq, d = q.shape
    num_pages, Hkv, page_size, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d] matching q")
    if page_table.shape[0] != B or ctx_lens.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and ctx_lens [B]")
    if scale is None:
        scale = d ** -0.5
    out = _out_like(out, q, "out")
    lse = _lse_out(lse, (B, H, Nq), q.device, return_lse)
    st = load_library().paged_attn_prefill_fp8(_dptr(q), _dptr(k_pages), _dptr(v_pages), float(k_scale),
                                               float(v_scale), _dptr(page_table), _dptr(ctx_lens), page_size,
                                               _dptr(out), _dptr(lse), B, H, Hkv, Nq, d, page_table.shape[1],
                                               num_pages, int(bool(causal)), float(scale), _stream_ptr(stream))
    _check("paged_attn_prefill_fp8", st)
    return out, lse


def paged_kv_append(k_new, v_new, k_pages, v_pages, page_table, start_pos, stream=None) -> None:
    """Write new tokens' K/V ([B,Hkv,Nnew,d] bf16) into the pages at positions start_pos[b] + t."""
    import torch
    _require(k_new, "k_new", torch.bfloat16, 4)
    _require(v_new, "v_new", torch.bfloat16, 4)
    _require(k_pages, "k_pages", torch.bfloat16, 4)
    _require(v_pages, "v_pages", torch.bfloat16, 4)
    _require(page_table, "page_table", torch.int32, 2)
    _require(start_pos, "start_pos", torch.int32, 1)
    B, Hkv, Nnew, d = k_new.shape
    num_pages, Hk, page_size, dk = k_pages.shape
    if (Hk, dk) != (Hkv, d) or tuple(v_new.shape) != tuple(k_new.shape) or tuple(v_pages.shape) != tuple(
            k_pages.shape):
        raise ValueError("shape mismatch between new K/V and the pages")
    st = load_library().paged_kv_append(_dptr(k_new), _dptr(v_new), _dptr(k_pages), _dptr(v_pages),
                                        _dptr(page_table), _dptr(start_pos), page_size, B, Hkv, Nnew, d,
                                        page_table.shape[1], num_pages, _stream_ptr(stream))
    _check("paged_kv_append", st)


def _torch():
    """torch, imported at the first call (the module itself loads without it), and with it the compiled
    marshalling if it was built against this torch."""
    global _t, _fast
    if _t is None:
        import torch
        lib = load_library()
        fast = _load_fastcall(torch.__version__, torch.compiled_with_cxx11_abi())
        if fast is not None:
            address = {n: ctypes.cast(getattr(lib, n), P).value for n in SIGNATURES}
            if fast.bind(address):
                _fast = fast
        _t = torch
    return _t


def _load_fastcall(torch_version, cxx11_abi):
    """The compiled marshalling built for this torch and this Python, or None."""
    from .build import fastcall_path
    path = fastcall_path(str(torch_version))
    if not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location(__package__ + "._fastcall", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
    except ImportError:
        return None
    return m if m.torch_version == str(torch_version) and bool(m.cxx11_abi) == bool(cxx11_abi) else None


_t = None
# Compiled marshalling (csrc/fastcall.cpp): each function takes the call's arguments and returns its
# result, the library's status, or None for a call that goes through the checks below.
_fast = None


def _in(t, name, dtype, ndim, device=None):
    """Address of a contiguous CUDA tensor of this dtype and number of dims on ``device`` (None: any).
    The checks of _require with one pass over the attributes: a call's host time counts where the
    kernel takes a few microseconds."""
    try:
        if t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
            if t.is_cuda and (device is None or t.device == device):
                return t.data_ptr()
    except AttributeError:
        pass
    _require(t, name, dtype, ndim)
    raise ValueError(f"{name} must be on {device}, got {t.device}")


def _elsewhere(device, stream):
    """Context that makes ``stream`` (None: the device's current stream) and its device current, or
    None if they already are.  Tensors allocated inside belong to that stream, so the allocator does
    not hand their memory to another stream's work while the call still uses it."""
    torch = _torch()
    if stream is None:
        return None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    return torch.cuda.stream(stream)


def _current_stream(device):
    return _t._C._cuda_getCurrentRawStream(device.index)


_Strides = ctypes.c_int64 * 3


def _rows_in(t, name, shape, device=None):
    """A [B, H, N, d] bf16 CUDA view with contiguous rows: its address and its strides as a C array
    (None if contiguous; the strides of dims of size one, which torch leaves arbitrary, count as 0)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    s = t.shape
    if len(s) != 4 or (shape is not None and s != shape):
        raise ValueError(f"{name} must be [B, heads, Nnew, d]" +
                         (f" = {tuple(shape)}" if shape is not None else "") + f", got {tuple(s)}")
    if t.is_contiguous():
        return t.data_ptr(), None
    b, h, n, e = t.stride()
    if e != 1:
        raise ValueError(f"the last dim of {name} must be contiguous")
    b, h, n = (0 if s[0] == 1 else b), (0 if s[1] == 1 else h), (0 if s[2] == 1 else n)
    if (b | h | n) & 7:
        raise ValueError(f"the strides of {name} must be multiples of 8 elements, got {t.stride()}")
    return t.data_ptr(), _Strides(b, h, n)


def _append_rope(fn, q, k_new, v_new, k_pages, v_pages, page_dtype, scales, cos_sin, page_table, start_pos,
                 interleaved, new_lens, q_out, stream):
    torch = _torch()
    kp, ks = _rows_in(k_new, "k_new", None)
    device = k_new.device
    B, Hkv, N, d = k_new.shape
    vp, vs = _rows_in(v_new, "v_new", k_new.shape, device)
    kpool, vpool = _in(k_pages, "k_pages", page_dtype, 4, device), _in(v_pages, "v_pages", page_dtype, 4, device)
    cs = _in(cos_sin, "cos_sin", torch.float32, 2, device)
    table = _in(page_table, "page_table", torch.int32, 2, device)
    start = _in(start_pos, "start_pos", torch.int32, 1, device)
    num_pages, Hk, page_size, dk = k_pages.shape
    if (Hk, dk) != (Hkv, d) or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, d] matching k_new")
    Bt, max_pages = page_table.shape
    if Bt != B or start_pos.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and start_pos [B]")
    new = None
    if new_lens is not None:
        new = _in(new_lens, "new_lens", torch.int32, 1, device)
        if new_lens.shape[0] != B:
            raise ValueError("new_lens must be [B]")
    H, qp, qs, qo = 0, None, None, None
    if q is not None:
        H = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 4 else 0
        qp, qs = _rows_in(q, "q", torch.Size((B, H, N, d)), device)
        if q_out is not None:
            qo = _in(q_out, "q_out", torch.bfloat16, 4, device)
            if q_out.shape != q.shape:
                raise ValueError(f"q_out must be {tuple(q.shape)}, got {tuple(q_out.shape)}")
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return _append_rope(fn, q, k_new, v_new, k_pages, v_pages, page_dtype, scales, cos_sin, page_table,
                                start_pos, interleaved, new_lens, q_out, None)
    if q is not None and q_out is None:
        q_out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=device)
        qo = q_out.data_ptr()
    st = getattr(load_library(), fn)(
        qp, qs, kp, ks, vp, vs, qo, kpool, vpool, *scales, cs, cos_sin.shape[1], cos_sin.shape[0], int(bool(interleaved)),
        table, start, new, page_size, B, H, Hkv, N, d, max_pages, num_pages, _current_stream(device))
    if st:
        _check(fn, st)
    return q_out


def _appended(fn, r):
    """The compiled append's answer: q_out, False (no query), or a status."""
    if r is False:
        return None
    if r.__class__ is int:
        _check(fn, r)
    return r


def paged_kv_append_rope(q, k_new, v_new, k_pages, v_pages, cos_sin, page_table, start_pos, interleaved: bool = False,
                         new_lens=None, q_out=None, stream=None):
    """Rotates new tokens' queries and keys to their positions and appends keys and values to the
    paged cache.  q [B,H,Nnew,d] (or None), k_new, v_new [B,Hkv,Nnew,d] bf16 CUDA views whose rows are
    contiguous (strides in multiples of 8 elements, so views of a fused projection need no copy);
    cos_sin [max_pos, rope_dim] fp32 (cos of the pairs, then sin); start_pos [B] int32; new_lens
    optional [B] int32, the tokens past it being padding, of which nothing is written (allocated
    q_out rows of padding are uninitialised).  Returns q_out [B,H,Nnew,d] bf16, contiguous (q itself
    may be given if contiguous)."""
    if _fast is not None and stream is None:
        r = _fast.append_rope(None, q, k_new, v_new, k_pages, v_pages, cos_sin, page_table, start_pos, interleaved,
                              new_lens, q_out)
        if r is not None:
            return _appended("paged_kv_append_rope", r)
    return _append_rope("paged_kv_append_rope", q, k_new, v_new, k_pages, v_pages, _torch().bfloat16, (), cos_sin,
                        page_table, start_pos, interleaved, new_lens, q_out, stream)


def paged_kv_append_rope_fp8(q, k_new, v_new, k_pages, v_pages, k_scale: float, v_scale: float, cos_sin, page_table,
                             start_pos, interleaved: bool = False, new_lens=None, q_out=None, stream=None):
    """paged_kv_append_rope into an e4m3 cache (k_pages, v_pages uint8 [P,Hkv,16,d])."""
    if _fast is not None and stream is None:
        r = _fast.append_rope((k_scale, v_scale), q, k_new, v_new, k_pages, v_pages, cos_sin, page_table, start_pos,
                              interleaved, new_lens, q_out)
        if r is not None:
            return _appended("paged_kv_append_rope_fp8", r)
    return _append_rope("paged_kv_append_rope_fp8", q, k_new, v_new, k_pages, v_pages, _torch().uint8,
                        (float(k_scale), float(v_scale)), cos_sin, page_table, start_pos, interleaved, new_lens,
                        q_out, stream)


def _optional(t, name, dtype, shape, device):
    """Address of an optional tensor of this shape (None if not given)."""
    if t is None:
        return None
    p = _in(t, name, dtype, len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return p


def _output(t, name, dtype, shape, device):
    """The output given by the caller (checked) or a new one: tensor and address."""
    if t is None:
        t = _t.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    p = _in(t, name, dtype, len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t, p


def _dense_inputs(q, k, v):
    """Addresses and sizes of q [B,Hq,Nq,d] and k, v [B,Hkv,Nkv,d], bf16 on one device."""
    bf = _torch().bfloat16
    qp = _in(q, "q", bf, 4)
    device = q.device
    kp, vp = _in(k, "k", bf, 4, device), _in(v, "v", bf, 4, device)
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nkv, dk = k.shape
    if Bk != B or dk != d or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, Nkv, d] matching q")
    return device, qp, kp, vp, B, Hq, Hkv, Nq, Nkv, d


def _scoremod_inputs(device, B, Hq, Nq, alibi_slopes, key_begin, key_end, kv_lens):
    i32 = _t.int32
    return (_optional(alibi_slopes, "alibi_slopes", _t.float32, (Hq,), device),
            _optional(key_begin, "key_begin", i32, (B, Nq), device),
            _optional(key_end, "key_end", i32, (B, Nq), device), _optional(kv_lens, "kv_lens", i32, (B,), device))


def attn_fwd_scoremod(q, k, v, causal: bool, scale: float | None = None, softcap: float = 0.0, alibi_slopes=None,
                      key_begin=None, key_end=None, kv_lens=None, out=None, lse=None, return_lse: bool = True,
                      stream=None):
    """Prefill with modified scores: softcap * tanh(scale q.k / softcap) - alibi_slopes[h] * |distance|
    over the keys key_begin[b,i] <= j < key_end[b,i] (and kv_lens, causal).  q [B,Hq,Nq,d], k/v
    [B,Hkv,Nkv,d] bf16; alibi_slopes [Hq] fp32; key_begin, key_end [B,Nq] int32; kv_lens [B] int32, all
    optional CUDA tensors; softcap 0 is none.  Returns (o, lse)."""
    if _fast is not None and stream is None:
        r = _fast.fwd_scoremod(q, k, v, causal, scale, softcap, alibi_slopes, key_begin, key_end, kv_lens, out, lse,
                               return_lse)
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check("attn_fwd_scoremod", r)
    device, qp, kp, vp, B, Hq, Hkv, Nq, Nkv, d = _dense_inputs(q, k, v)
    mod = _scoremod_inputs(device, B, Hq, Nq, alibi_slopes, key_begin, key_end, kv_lens)
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return attn_fwd_scoremod(q, k, v, causal, scale, softcap, alibi_slopes, key_begin, key_end, kv_lens, out,
                                     lse, return_lse)
    out, op = _output(out, "out", _t.bfloat16, (B, Hq, Nq, d), device)
    lp = None
    if lse is not None or return_lse:
        lse, lp = _output(lse, "lse", _t.float32, (B, Hq, Nq), device)
    st = load_library().attn_fwd_scoremod(qp, kp, vp, op, lp, B, Hq, Hkv, Nq, Nkv, d, int(bool(causal)),
                                          d ** -0.5 if scale is None else scale, softcap, *mod,
                                          _current_stream(device))
    if st:
        _check("attn_fwd_scoremod", st)
    return out, lse


def attn_bwd_scoremod_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, Nkv: int, d: int) -> int:
    return int(load_library().attn_bwd_scoremod_workspace_size(B, Hq, Hkv, Nq, Nkv, d))


def _workspace(t, need, device):
    """The caller's uint8 workspace (its size is checked by the library) or a new one: tensor, address, bytes."""
    if t is None:
        t = _t.empty(need if need > 16 else 16, dtype=_t.uint8, device=device)
        return t, t.data_ptr(), t.numel()
    return t, _in(t, "workspace", _t.uint8, 1, device), t.numel()


def attn_bwd_scoremod(q, k, v, o, lse, dout, causal: bool, scale: float | None = None, softcap: float = 0.0,
                      alibi_slopes=None, key_begin=None, key_end=None, kv_lens=None, dq=None, dk=None, dv=None,
                      workspace=None, stream=None):
    """Backward of attn_fwd_scoremod: q, o, dout [B,Hq,Nq,d] and k, v [B,Hkv,Nkv,d] bf16, lse [B,Hq,Nq]
    fp32 from the forward, the modification as in the forward call.  Returns (dq, dk, dv) bf16.
    workspace: optional uint8 tensor of attn_bwd_scoremod_workspace_size(B, Hq, Hkv, Nq, Nkv, d) bytes."""
    if _fast is not None and stream is None:
        r = _fast.bwd_scoremod(q, k, v, o, lse, dout, causal, scale, softcap, alibi_slopes, key_begin, key_end, kv_lens,
                               dq, dk, dv, workspace)
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check("attn_bwd_scoremod", r)
    device, qp, kp, vp, B, Hq, Hkv, Nq, Nkv, d = _dense_inputs(q, k, v)
    bf = _t.bfloat16
    op, lp = _in(o, "o", bf, 4, device), _in(lse, "lse", _t.float32, 3, device)
    gp = _in(dout, "dout", bf, 4, device)
    if o.shape != q.shape or dout.shape != q.shape or lse.shape != q.shape[:3]:
        raise ValueError("o and dout must match q, lse must be [B, Hq, Nq]")
    mod = _scoremod_inputs(device, B, Hq, Nq, alibi_slopes, key_begin, key_end, kv_lens)
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return attn_bwd_scoremod(q, k, v, o, lse, dout, causal, scale, softcap, alibi_slopes, key_begin, key_end,
                                     kv_lens, dq, dk, dv, workspace)
    dq, dqp = _output(dq, "dq", bf, q.shape, device)
    dk, dkp = _output(dk, "dk", bf, k.shape, device)
    dv, dvp = _output(dv, "dv", bf, k.shape, device)
    lib = load_library()
    workspace, wp, wn = _workspace(workspace, lib.attn_bwd_scoremod_workspace_size(B, Hq, Hkv, Nq, Nkv, d), device)
    st = lib.attn_bwd_scoremod(qp, kp, vp, op, lp, gp, dqp, dkp, dvp, B, Hq, Hkv, Nq, Nkv, d, int(bool(causal)),
                               d ** -0.5 if scale is None else scale, softcap, *mod, wp, wn, _current_stream(device))
    if st:
        _check("attn_bwd_scoremod", st)
    return dq, dk, dv


def paged_attn_decode_scoremod_workspace_size(B: int, H: int, Hkv: int, d: int, max_pages_per_seq: int,
                                              page_size: int = 16) -> int:
    return int(load_library().paged_attn_decode_scoremod_workspace_size(B, H, Hkv, d, max_pages_per_seq, page_size))


def paged_attn_decode_shared_workspace_size(B: int, H: int, Hkv: int, d: int, max_pages_per_seq: int,
                                            group_size: int, page_size: int = 16) -> int:
    return int(load_library().paged_attn_decode_shared_workspace_size(B, H, Hkv, d, max_pages_per_seq, group_size,
                                                                      page_size))


def _paged_inputs(q, k_pages, v_pages, page_dtype, page_table, ctx_lens):
    """Addresses and sizes of a decode batch over a paged cache, on one device."""
    torch = _torch()
    qp = _in(q, "q", torch.bfloat16, 3)
    device = q.device
    kp, vp = _in(k_pages, "k_pages", page_dtype, 4, device), _in(v_pages, "v_pages", page_dtype, 4, device)
    table, ctx = _in(page_table, "page_table", torch.int32, 2, device), _in(ctx_lens, "ctx_lens", torch.int32, 1, device)
    B, H, d = q.shape
    num_pages, Hkv, page_size, dk = k_pages.shape
    if dk != d or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d] matching q")
    Bt, max_pages = page_table.shape
    if Bt != B or ctx_lens.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages] and ctx_lens [B]")
    return device, (qp, kp, vp, table, ctx), (B, H, Hkv, d, max_pages, num_pages), page_size


def _decode_outputs(out, lse, return_lse, B, H, d, device):
    out, op = _output(out, "out", _t.bfloat16, (B, H, d), device)
    lp = None
    if lse is not None or return_lse:
        lse, lp = _output(lse, "lse", _t.float32, (B, H), device)
    return out, op, lse, lp


def _decode_scoremod(fn, page_dtype, scales, q, k_pages, v_pages, page_table, ctx_lens, scale, softcap, alibi_slopes,
                     key_begin, out, lse, workspace, return_lse, stream):
    if _fast is not None and stream is None:
        r = _fast.decode_scoremod(scales or None, q, k_pages, v_pages, page_table, ctx_lens, scale, softcap,
                                  alibi_slopes, key_begin, out, lse, workspace, return_lse)
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(fn, r)
    device, (qp, kp, vp, table, ctx_p), sizes, ps = _paged_inputs(q, k_pages, v_pages, page_dtype, page_table, ctx_lens)
    B, H, Hkv, d, max_pages, num_pages = sizes
    slopes = _optional(alibi_slopes, "alibi_slopes", _t.float32, (H,), device)
    begin = _optional(key_begin, "key_begin", _t.int32, (B,), device)
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return _decode_scoremod(fn, page_dtype, scales, q, k_pages, v_pages, page_table, ctx_lens, scale, softcap,
                                    alibi_slopes, key_begin, out, lse, workspace, return_lse, None)
    out, op, lse, lp = _decode_outputs(out, lse, return_lse, B, H, d, device)
    lib = load_library()
    workspace, wp, wn = _workspace(
        workspace, lib.paged_attn_decode_scoremod_workspace_size(B, H, Hkv, d, max_pages, ps), device)
    st = getattr(lib, fn)(qp, kp, vp, *scales, table, ctx_p, ps, op, lp, *sizes, d ** -0.5 if scale is None else scale,
                          softcap, slopes, begin, wp, wn, _current_stream(device))
    if st:
        _check(fn, st)
    return out, lse


def paged_attn_decode_scoremod(q, k_pages, v_pages, page_table, ctx_lens, scale: float | None = None,
                               softcap: float = 0.0, alibi_slopes=None, key_begin=None, out=None, lse=None,
                               workspace=None, return_lse: bool = True, stream=None):
    """Paged decode with modified scores: softcap * tanh(scale q.k / softcap) - alibi_slopes[h] * distance over
    the cached tokens key_begin[b] <= j < ctx_lens[b].  q [B,H,d] bf16; k_pages/v_pages [P,Hkv,16,d] bf16;
    page_table [B,max_pages], ctx_lens [B] int32; alibi_slopes [H] fp32 and key_begin [B] int32 optional;
    softcap 0 is none.  Returns (o, lse)."""
    return _decode_scoremod("paged_attn_decode_scoremod", _torch().bfloat16, (), q, k_pages, v_pages, page_table,
                            ctx_lens, scale, softcap, alibi_slopes, key_begin, out, lse, workspace, return_lse, stream)


def paged_attn_decode_scoremod_fp8(q, k_pages, v_pages, k_scale: float, v_scale: float, page_table, ctx_lens,
                                   scale: float | None = None, softcap: float = 0.0, alibi_slopes=None,
                                   key_begin=None, out=None, lse=None, workspace=None, return_lse: bool = True,
                                   stream=None):
    """paged_attn_decode_scoremod over an e4m3 cache (k_pages, v_pages uint8 codes [P,Hkv,16,d])."""
    return _decode_scoremod("paged_attn_decode_scoremod_fp8", _torch().uint8, (float(k_scale), float(v_scale)), q,
                            k_pages, v_pages, page_table, ctx_lens, scale, softcap, alibi_slopes, key_begin, out, lse,
                            workspace, return_lse, stream)


def _decode_shared(fn, page_dtype, scales, q, k_pages, v_pages, page_table, ctx_lens, shared_pages, group_size, scale,
                   out, lse, workspace, return_lse, stream):
    if _fast is not None and stream is None:
        r = _fast.decode_shared(scales or None, q, k_pages, v_pages, page_table, ctx_lens, shared_pages, group_size,
                                scale, out, lse, workspace, return_lse)
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(fn, r)
    device, (qp, kp, vp, table, ctx_p), sizes, ps = _paged_inputs(q, k_pages, v_pages, page_dtype, page_table, ctx_lens)
    B, H, Hkv, d, max_pages, num_pages = sizes
    if group_size <= 0 or B % group_size:
        raise ValueError(f"the batch of {B} must be whole groups of group_size = {group_size} sequences")
    shared = _optional(shared_pages, "shared_pages", _t.int32, (B // group_size,), device)
    if shared is None:
        raise TypeError("shared_pages must be a torch.Tensor")
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return _decode_shared(fn, page_dtype, scales, q, k_pages, v_pages, page_table, ctx_lens, shared_pages,
                                  group_size, scale, out, lse, workspace, return_lse, None)
    out, op, lse, lp = _decode_outputs(out, lse, return_lse, B, H, d, device)
    lib = load_library()
    workspace, wp, wn = _workspace(
        workspace, lib.paged_attn_decode_shared_workspace_size(B, H, Hkv, d, max_pages, group_size, ps), device)
    st = getattr(lib, fn)(qp, kp, vp, *scales, table, ctx_p, shared, group_size, ps, op, lp, *sizes,
                          d ** -0.5 if scale is None else scale, wp, wn, _current_stream(device))
    if st:
        _check(fn, st)
    return out, lse


def paged_attn_decode_shared(q, k_pages, v_pages, page_table, ctx_lens, shared_pages, group_size: int,
                             scale: float | None = None, out=None, lse=None, workspace=None, return_lse: bool = True,
                             stream=None):
    """Paged decode of groups of group_size consecutive sequences that share their first pages, which are read
    once per group: q [B,H,d] bf16; k_pages/v_pages [P,Hkv,16,d] bf16; page_table [B,max_pages], ctx_lens [B]
    int32; shared_pages [B/group_size] int32, the number of shared page-table entries of each group (taken from
    its first sequence's row).  Returns (o, lse)."""
    return _decode_shared("paged_attn_decode_shared", _torch().bfloat16, (), q, k_pages, v_pages, page_table, ctx_lens,
                          shared_pages, group_size, scale, out, lse, workspace, return_lse, stream)


def paged_attn_decode_shared_fp8(q, k_pages, v_pages, k_scale: float, v_scale: float, page_table, ctx_lens,
                                 shared_pages, group_size: int, scale: float | None = None, out=None, lse=None,
                                 workspace=None, return_lse: bool = True, stream=None):
    """paged_attn_decode_shared over an e4m3 cache (k_pages, v_pages uint8 codes [P,Hkv,16,d])."""
    return _decode_shared("paged_attn_decode_shared_fp8", _torch().uint8, (float(k_scale), float(v_scale)), q, k_pages,
                          v_pages, page_table, ctx_lens, shared_pages, group_size, scale, out, lse, workspace,
                          return_lse, stream)


def attn_selftest_bounded_wait(stream=None) -> None:
    """Launch the bounded-wait self-test kernel (its wait runs out after about 2 s)."""
    _check("attn_selftest_bounded_wait", load_library().attn_selftest_bounded_wait(_stream_ptr(stream)))


def attn_check_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the library's device status word."""
    return int(load_library().attn_check_device_status(_stream_ptr(stream)))


def attn_last_device_status() -> int:
    """The current device's host-visible timeout flag, without synchronising or clearing."""
    return int(load_library().attn_last_device_status())
