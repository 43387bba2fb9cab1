"""Thin Python binding of ``libattn_gb300.so`` (ctypes): argument marshalling only.

Every step of the attention forward runs in the library's CUDA kernels; PyTorch only supplies
device memory, streams and the output allocations.  There is no fallback: if the library is
missing or the GPU is not an sm_103 part, calls raise.

Layouts (same as the C ABI in ``include/attn_gb300.h``):
  dense  q, k, v, o: [B, H, N, d] bf16 contiguous; lse [B, H, N] fp32
  packed q, k, v, o: [H, T, d] bf16 contiguous + cu_seqlens int32 [n+1]; lse [H, T] fp32
  paged  K, V caches: [num_pages, H_kv, page_size, d] bf16 or E4M3 (see KVCache)
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Any, NamedTuple

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn_gb300.so")

STATUS = {
    0: "ATTN_OK", -1: "ATTN_ERR_NULL", -2: "ATTN_ERR_HEAD_DIM", -3: "ATTN_ERR_SHAPE",
    -4: "ATTN_ERR_ALIGN", -5: "ATTN_ERR_LAUNCH", -6: "ATTN_ERR_DEVICE", -7: "ATTN_ERR_SCALE",
    -8: "ATTN_ERR_WORKSPACE", -9: "ATTN_ERR_UNSUPPORTED", -10: "ATTN_ERR_SCRATCH_LIMIT",
}

# exported C symbols and their ctypes signatures (kept in step with include/attn_gb300.h)
_P, _I, _F, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L = ctypes.c_int64
SIGNATURES = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "attn_fwd_gqa": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "attn_fwd_splitkv": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _S, _P]),
    "attn_fwd_splitkv_workspace_bytes": (_S, [_I, _I, _I, _I, _I]),
    "attn_fwd_splitkv_slices": (_I, [_I, _I, _I, _I, _I]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _S, _P]),
    "attn_bwd_gqa": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P,
                          _S, _P]),
    "attn_bwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                             _F, _P, _S, _P]),
    "attn_bwd_varlen_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "attn_bwd_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "attn_quantize_fp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "attn_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "attn_kv_slots": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "attn_qkv_rope": (_I, [_P, _L, _P, _P, _F, _P, _I, _I, _F, _P, _P, _P, _P, _P, _P, _I, _I, _I,
                           _I, _I, _P]),
    "attn_qkv_rope_bwd": (_I, [_P, _P, _P, _P, _L, _P, _P, _F, _P, _I, _I, _F, _P, _P, _L, _P, _P,
                               _I, _I, _I, _I, _I, _P, _S, _P]),
    "attn_qkv_rope_bwd_workspace_bytes": (_S, [_I, _I, _I, _I, _I]),
    "attn_fwd_paged": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _S, _P]),
    "attn_fwd_paged_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "attn_fwd_paged_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _S, _P]),
    "attn_fwd_paged_varlen_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "attn_fwd_paged_shared": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                   _S, _P]),
    "attn_fwd_paged_shared_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "attn_kv_write": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "attn_kv_read": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "attn_fwd_unfused": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _S, _P]),
    "attn_fwd_unfused_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "attn_fwd_unfused_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "attn_get_last_device_error": (_I, [_P]),
    "attn_selftest_mma": (_I, [_P, _P, _P, _I, _I, _P]),
    "attn_selftest_wait_timeout": (_I, [_P]),
    "attn_selftest_fp8_quotients": (_I, [_P, _P]),
    "attn_version": (_I, []),
}


class AttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({code})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m io_aware_attention_attn_gb300.build`"
                " (or __graft_entry__.build())")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _lib = handle
    return _lib


def _check(name: str, rc: int):
    if rc != 0:
        raise AttnError(name, rc)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_inputs(q, k, v, cu_seqlens, allow_kv_heads=False):
    """Returns (B, H, H_kv, N, d).  K and V may have fewer heads than Q when allow_kv_heads."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
        if t.dim() != q.dim() or t.device != q.device:
            raise ValueError("q, k and v must have the same rank and device")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    hd = 1 if cu_seqlens is None else 0  # index of the head axis
    if q.shape[:hd] + q.shape[hd + 1:] != k.shape[:hd] + k.shape[hd + 1:]:
        raise ValueError("q and k/v differ in a dimension other than heads")
    if not allow_kv_heads and k.shape != q.shape:
        raise ValueError("q, k and v must have the same shape")
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("dense inputs are [B, H, N, d]")
        B, H, N, d = q.shape
    else:
        if q.dim() != 3:
            raise ValueError("packed inputs are [H, T, d] with cu_seqlens")
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or \
                not cu_seqlens.is_contiguous() or cu_seqlens.dim() != 1 or \
                cu_seqlens.device != q.device:
            raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor on q's device")
        H, N, d = q.shape
        B = cu_seqlens.numel() - 1
    H_kv = k.shape[hd]
    if H_kv == 0 or H % H_kv != 0:
        raise ValueError("the number of K/V heads must divide the number of query heads")
    return B, H, H_kv, N, d


def attn_fwd(q, k, v, cu_seqlens=None, causal: bool = False, scale: float | None = None,
             out=None, lse=None, stream=None):
    """Fused attention forward.  Returns (O bf16 like q, LSE fp32).

    k and v may have fewer heads than q (grouped-query / multi-query attention: query head h
    reads K/V head h // (H // H_kv)); then the attn_fwd_gqa entry point is called."""
    import torch
    B, H, H_kv, N, d = _check_inputs(q, k, v, cu_seqlens, allow_kv_heads=True)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    cu = cu_seqlens.data_ptr() if cu_seqlens is not None else None
    with torch.cuda.device(q.device):
        st = _stream_handle(stream, q.device)
        if H_kv == H:
            rc = lib().attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                lse.data_ptr(), cu, B, H, N, d, int(bool(causal)), float(scale), st)
        else:
            rc = lib().attn_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), cu, B, H, H_kv, N, d, int(bool(causal)),
                                    float(scale), st)
    _check("attn_fwd_gqa" if H_kv != H else "attn_fwd", rc)
    return out, lse


def splitkv_workspace_bytes(B: int, H: int, N: int, d: int, num_splits: int = 0) -> int:
    return int(lib().attn_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits))


def splitkv_slices(B: int, H: int, N: int, d: int, num_splits: int = 0) -> int:
    return int(lib().attn_fwd_splitkv_slices(B, H, N, d, num_splits))


def attn_fwd_splitkv(q, k, v, causal: bool = False, scale: float | None = None,
                     num_splits: int = 0, workspace=None, out=None, lse=None, stream=None):
    """Split-KV fused forward (dense [B, H, N, d] only): the key range of every query pair is
    cut into ``num_splits`` slices (0: the library chooses) whose partial results a second kernel
    merges.  Returns (O bf16 like q, LSE fp32)."""
    import torch
    B, H, _, N, d = _check_inputs(q, k, v, None)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = splitkv_workspace_bytes(B, H, N, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                                    int(num_splits), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(),
                                    _stream_handle(stream, q.device))
    _check("attn_fwd_splitkv", rc)
    return out, lse


def bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, H, N, d))


def attn_bwd(q, k, v, o, lse, dout, cu_seqlens=None, causal: bool = False,
             scale: float | None = None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Backward pass: gradients (dQ, dK, dV) of the fused forward for the upstream gradient
    ``dout``, given the forward's ``o`` and ``lse``.  Dense [B, H, N, d], or packed [H, T, d] with
    ``cu_seqlens`` (attn_bwd_varlen); k and v may have fewer heads than q (grouped-query: dK and dV
    summed over each group)."""
    import torch
    B, H, H_kv, N, d = _check_inputs(q, k, v, cu_seqlens, allow_kv_heads=True)
    for name, t in (("o", o), ("dout", dout)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or t.shape != q.shape or \
                t.device != q.device:
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like q")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != q.shape[:-1] or \
            lse.device != q.device:
        raise ValueError("lse must be a contiguous fp32 tensor of shape [B, H, N]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = (bwd_workspace_bytes(B, H, N, d) if cu_seqlens is None
            else int(lib().attn_bwd_varlen_workspace_bytes(B, H, N, d)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws = (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    with torch.cuda.device(q.device):
        st = _stream_handle(stream, q.device)
        if cu_seqlens is not None:
            rc = lib().attn_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                       lse.data_ptr(), dout.data_ptr(), dq.data_ptr(),
                                       dk.data_ptr(), dv.data_ptr(), cu_seqlens.data_ptr(), B, H,
                                       H_kv, N, d, int(bool(causal)), float(scale), *ws, st)
        elif H_kv == H:
            rc = lib().attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), B, H, N, d, int(bool(causal)), float(scale), *ws, st)
        else:
            rc = lib().attn_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                    lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                    dv.data_ptr(), B, H, H_kv, N, d, int(bool(causal)),
                                    float(scale), *ws, st)
    _check("attn_bwd_varlen" if cu_seqlens is not None else
           ("attn_bwd_gqa" if H_kv != H else "attn_bwd"), rc)
    return dq, dk, dv


def quantize_fp8(x, transpose: bool = False, stream=None):
    """Per-tile E4M3 quantization of a dense bf16 tensor [B, H, N, d].  Returns (codes uint8,
    scales fp32 [B, H, ceil(N/128)]); codes are [B, H, N, d], or [B, H, d, Npad] when
    ``transpose`` (the V operand of attn_fwd_fp8)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 4:
        raise ValueError("x must be a contiguous [B, H, N, d] bf16 CUDA tensor")
    B, H, N, d = x.shape
    T = -(-N // 128)
    shape = (B, H, d, T * 128) if transpose else (B, H, N, d)
    codes = torch.empty(shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((B, H, T), dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        rc = lib().attn_quantize_fp8(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), B, H, N,
                                     d, int(bool(transpose)), _stream_handle(stream, x.device))
    _check("attn_quantize_fp8", rc)
    return codes, scales


def attn_fwd_fp8(q8, sq, k8, sk, vt8, sv, causal: bool = False, scale: float | None = None,
                 out=None, lse=None, stream=None):
    """FP8 fused forward on quantized inputs (see quantize_fp8).  Returns (O bf16, LSE fp32)."""
    import torch
    if q8.dtype != torch.uint8 or q8.dim() != 4 or not q8.is_contiguous():
        raise ValueError("q8 must be contiguous [B, H, N, 128] uint8 codes")
    B, H, N, d = q8.shape
    T = -(-N // 128)
    if k8.shape != q8.shape or vt8.shape != (B, H, d, T * 128) or \
            sq.shape != (B, H, T) or sk.shape != (B, H, T) or sv.shape != (B, H, T):
        raise ValueError("k8, vt8 and the scales must match q8 (vt8 is [B, H, d, Npad])")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    with torch.cuda.device(q8.device):
        rc = lib().attn_fwd_fp8(q8.data_ptr(), sq.data_ptr(), k8.data_ptr(), sk.data_ptr(),
                                vt8.data_ptr(), sv.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, H, N, d, int(bool(causal)), float(scale),
                                _stream_handle(stream, q8.device))
    _check("attn_fwd_fp8", rc)
    return out, lse


# ------------------------------------------------------------------------------- generation
class KVCache(NamedTuple):
    """A paged key-value cache: k, v [num_pages, H_kv, page_size, d], bf16, or E4M3 codes
    (torch.float8_e4m3fn or uint8) with k_scale, v_scale fp32 [num_pages, H_kv, page_size].  The stride
    from page to page is free (k and v may be the two halves of one tensor of pages); inside a
    page the rows are contiguous."""
    k: Any
    v: Any
    k_scale: Any = None
    v_scale: Any = None


def kv_cache(num_pages: int, H_kv: int, page_size: int, d: int, dtype=None, device="cuda") -> KVCache:
    """An empty cache (zeros): bf16, or E4M3 with dtype torch.float8_e4m3fn."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8):
        raise ValueError("a cache is bf16 or float8_e4m3fn")
    shape = (num_pages, H_kv, page_size, d)
    kind = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
    k, v = (torch.zeros(shape, dtype=kind, device=device).view(dtype) for _ in range(2))
    if dtype == torch.bfloat16:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device)
                           for _ in range(2)))


_native_module = None


def _native():
    """The marshalling module of the generation path (csrc/py_binding.cpp), loaded once.  Its
    functions check the tensors, allocate the outputs and call the C entry point on the current stream of
    the tensors' device; in Python and ctypes that took several times as long as these kernels."""
    global _native_module
    if _native_module is None:
        lib()
        from . import build
        if not build.binding_matches():  # it takes torch's objects apart: no call into another layout
            raise RuntimeError(
                f"{build.BINDING} is missing or was built for another torch or Python than this one: build it "
                "with `python -m io_aware_attention_attn_gb300.build`")
        from . import _attn_binding
        _attn_binding.set_error(AttnError)
        _native_module = _attn_binding
    return _native_module


def _on(stream, device):
    """Makes ``stream`` (a torch stream or a cudaStream_t) current: torch's allocations of the call
    are then made on it, and a buffer released after the call is not handed out before its work is
    done."""
    import torch
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
            torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def kv_slots(seq_lens, cu_new, T: int, block_table, free_pages, free_head, page_size: int,
             stream=None):
    """Pages, slots and positions of T new tokens (see attn_kv_slots in the header).  seq_lens
    int32 [B], cu_new int32 [B + 1], block_table int32 [B, max_pages] (new entries are written),
    free_pages int32 [n], free_head int32 [1].  Returns (slots int64 [T], positions int32 [T],
    block_table, new seq_lens, new free_head); the old seq_lens and free_head are left alone.
    A request may hold tokens and get several more: attn_fwd_paged_varlen attends for those.
    Slots and positions share one storage, and so do lengths and head (all four at up to one new token a
    request): clone what is saved or handed to another process by itself."""
    if stream is not None:
        with _on(stream, seq_lens.device):
            return kv_slots(seq_lens, cu_new, T, block_table, free_pages, free_head, page_size)
    return _native().kv_slots(seq_lens, cu_new, T, block_table, free_pages, free_head, page_size)


def rope_inv_freq(rot: int, base: float = 10000.0, factor: float = 1.0, original_len: int = 0,
                  low: float = 1.0, high: float = 4.0, device="cuda"):
    """Rotation frequencies base^(-2i/rot), float64 [rot/2], radians a position.  factor > 1
    stretches them for a longer context: all of them divided by it, or, with original_len, only those
    that turn fewer than ``low`` times over original_len positions, none of those that turn
    more than ``high`` times, and a linear blend between."""
    import torch
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    if factor != 1.0:
        if original_len:
            turns = original_len * f / (2.0 * math.pi)
            keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
            f = f * (keep + (1.0 - keep) / factor)
        else:
            f = f / factor
    return f.to(device)


_NO_CACHE = KVCache(None, None)


def qkv_rope(qkv, H: int, H_kv: int, positions=None, inv_freq=None, interleaved: bool = False,
             wq=None, wk=None, eps: float = 1e-6, rope_scale: float = 1.0, cache=None, slots=None,
             with_kv: bool = True, stream=None):
    """q, k, v of a projection's rows: RMS norm of each query and key head where wq, wk (bf16 [d])
    are given, rotation of the first 2 len(inv_freq) elements by positions (int32, shaped like the
    rows), head-major layout.  qkv [B, N, (H + 2 H_kv) d] gives q [B, H, N, d] and k, v
    [B, H_kv, N, d] (attn_fwd dense; attn_fwd_paged for N = 1); qkv [T, ...] gives the packed
    [H, T, d].  With ``cache`` the K and V rows also go to ``slots`` (int64, shaped like the rows;
    negative: not stored).  with_kv=False returns None for k and v."""
    if stream is not None:
        with _on(stream, qkv.device):
            return qkv_rope(qkv, H, H_kv, positions, inv_freq, interleaved, wq, wk, eps,
                            rope_scale, cache, slots, with_kv)
    return _native().qkv_rope(qkv, H, H_kv, positions, inv_freq, interleaved, wq, wk, eps, rope_scale,
                              *(cache or _NO_CACHE), slots, with_kv)


def qkv_rope_bwd(dq, dk, dv, qkv, positions=None, inv_freq=None, interleaved: bool = False, wq=None,
                 wk=None, eps: float = 1e-6, rope_scale: float = 1.0, workspace=None, stream=None):
    """Backward of qkv_rope: the gradient of qkv's rows (contiguous, qkv's shape) from dq [B, H, N, d]
    (or [H, T, d]) and dk, dv, and fp32 gradients of wq and wk (None where not given), the two halves
    of one storage."""
    if stream is not None:
        with _on(stream, qkv.device):
            return qkv_rope_bwd(dq, dk, dv, qkv, positions, inv_freq, interleaved, wq, wk, eps,
                                rope_scale, workspace)
    return _native().qkv_rope_bwd(dq, dk, dv, qkv, positions, inv_freq, interleaved, wq, wk, eps,
                                  rope_scale, workspace)


def paged_workspace_bytes(B: int, H: int, H_kv: int, d: int) -> int:
    return int(lib().attn_fwd_paged_workspace_bytes(B, H, H_kv, d))


def attn_fwd_paged(q, cache, block_table, seq_lens, scale: float | None = None, workspace=None,
                   out=None, lse=None, stream=None):
    """Attention of one new token of each request over a paged cache: q [B, H, 1, d] (or [B, H, d]),
    block_table int32 [B, max_pages], seq_lens int32 [B] (rows in the cache, the new token's own
    among them).  Returns (O bf16 like q, LSE fp32 [B, H, 1] or [B, H])."""
    if stream is not None:
        with _on(stream, q.device):
            return attn_fwd_paged(q, cache, block_table, seq_lens, scale, workspace, out, lse)
    return _native().attn_fwd_paged(q, *cache, block_table, seq_lens, scale, workspace, out, lse)


def paged_varlen_workspace_bytes(T: int, H: int, H_kv: int, d: int) -> int:
    return int(lib().attn_fwd_paged_varlen_workspace_bytes(T, H, H_kv, d))


def attn_fwd_paged_varlen(q, cache, block_table, seq_lens, cu_new, causal: bool = True,
                          scale: float | None = None, workspace=None, out=None, lse=None, stream=None):
    """Attention of several new tokens of each request over a paged cache: q [H, T, d] packed by cu_new int32
    [B + 1], block_table int32 [B, max_pages], seq_lens int32 [B] (rows in the cache, the new tokens'
    own among them).  Token i of a request's n sees rows 0 .. seq_lens - n + i, or all of them with
    causal=False.  Returns (O bf16 like q, LSE fp32 [H, T]); tokens from cu_new[B] on are padding, their
    rows are left as they were in ``out`` and ``lse`` (unspecified where those are not given)."""
    if stream is not None:
        with _on(stream, q.device):
            return attn_fwd_paged_varlen(q, cache, block_table, seq_lens, cu_new, causal, scale, workspace, out, lse)
    return _native().attn_fwd_paged_varlen(q, *cache, block_table, seq_lens, cu_new, causal, scale, workspace, out,
                                           lse)


def paged_shared_workspace_bytes(B: int, H: int, H_kv: int, d: int) -> int:
    return int(lib().attn_fwd_paged_shared_workspace_bytes(B, H, H_kv, d))


def attn_fwd_paged_shared(q, cache, prefix_table, prefix_lens, cu_groups, block_table, seq_lens,
                          scale: float | None = None, workspace=None, out=None, lse=None, stream=None):
    """attn_fwd_paged for requests that share their first rows, which are read once for all of a group:
    requests cu_groups[g] .. cu_groups[g+1]-1 (int32 [groups + 1]) have the prefix_lens[g] rows of the pages
    prefix_table[g] (int32 [groups, max_prefix_pages]) before the seq_lens rows of their own pages block_table.
    q [B, H, 1, d] (or [B, H, d]).  Returns (O bf16 like q, LSE fp32 [B, H, 1] or [B, H])."""
    if stream is not None:
        with _on(stream, q.device):
            return attn_fwd_paged_shared(q, cache, prefix_table, prefix_lens, cu_groups, block_table, seq_lens, scale,
                                         workspace, out, lse)
    return _native().attn_fwd_paged_shared(q, *cache, prefix_table, prefix_lens, cu_groups, block_table, seq_lens,
                                           scale, workspace, out, lse)


def kv_write(k, v, cache, slots, stream=None):
    """K and V rows into the cache at ``slots`` (int64; negative: not stored), without norm or rotation: k, v
    [B, H_kv, N, d] with slots [B, N], or [H_kv, T, d] with slots [T]; any strides that keep rows of d
    contiguous (a projection's token-major rows, transposed, are fine).  E4M3 caches get codes
    and scales as from qkv_rope.  Returns the cache."""
    if stream is not None:
        with _on(stream, k.device):
            return kv_write(k, v, cache, slots)
    _native().kv_write(k, v, *cache, slots)
    return cache


def kv_read(cache, block_table, cu_rows, T: int, first=None, out_k=None, out_v=None, stream=None):
    """Rows of the cache's requests as packed bf16 k, v [H_kv, T, d] (what attn_fwd takes): row
    cu_rows[s] + i is row first[s] + i (first int32 [B]; None: from the beginning) of request s's pages
    block_table[s].  Rows from cu_rows[B] on are left as they were in ``out_k`` and ``out_v``."""
    if stream is not None:
        with _on(stream, cache.k.device):
            return kv_read(cache, block_table, cu_rows, T, first, out_k, out_v)
    return _native().kv_read(*cache, block_table, cu_rows, T, first, out_k, out_v)


def unfused_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().attn_fwd_unfused_workspace_bytes(B, H, N, d))


def attn_fwd_unfused(q, k, v, causal: bool = False, scale: float | None = None, workspace=None,
                     out=None, lse=None, stream=None):
    """Unfused three-kernel comparison path (S and P through HBM).  Dense layout only."""
    import torch
    B, H, _, N, d = _check_inputs(q, k, v, None)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = unfused_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_unfused(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), None, B, H, N, d, int(bool(causal)),
                                    float(scale), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(),
                                    _stream_handle(stream, q.device))
    _check("attn_fwd_unfused", rc)
    return out, lse


def attn_fwd_unfused_noalloc(q, k, v, causal: bool = False, scale: float | None = None,
                             out=None, lse=None, stream=None):
    """The unfused path using the library's built-in scratch instead of a workspace (for callers
    that cannot allocate device memory; outputs may still be allocated here when not given)."""
    import torch
    B, H, _, N, d = _check_inputs(q, k, v, None)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_unfused_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            out.data_ptr(), lse.data_ptr(), B, H, N, d,
                                            int(bool(causal)), float(scale),
                                            _stream_handle(stream, q.device))
    _check("attn_fwd_unfused_noalloc", rc)
    return out, lse


def last_device_error(stream=None, device=None) -> int:
    """Device status word of the kernels on ``stream`` (0 = every pipeline wait completed)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        rc = lib().attn_get_last_device_error(_stream_handle(stream, dev))
    if rc < 0:
        raise AttnError("attn_get_last_device_error", rc)
    return rc


def selftest_mma(a, b, mode: int):
    """Diagnostic single-tile tensor-core product (see attn_selftest_mma in the header)."""
    import torch
    dim = b.shape[1]
    n_out = 128 if mode == 0 else dim
    d = torch.empty((128, n_out), dtype=torch.float32, device=a.device)
    with torch.cuda.device(a.device):
        rc = lib().attn_selftest_mma(a.data_ptr(), b.data_ptr(), d.data_ptr(), mode, dim,
                                     _stream_handle(None, a.device))
    _check("attn_selftest_mma", rc)
    return d


def selftest_wait_timeout(stream=None):
    """Launch the bounded-wait self-test (returns at once; the status appears after ~1 s)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device())
    _check("attn_selftest_wait_timeout",
           lib().attn_selftest_wait_timeout(_stream_handle(stream, dev)))


def selftest_fp8_quotients(stream=None) -> int:
    """Pairs (x, tile maximum) whose quantizer code differs from the code of the IEEE quotient
    (see attn_selftest_fp8_quotients in the header); synchronises the stream."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device())
    out = torch.zeros(1, dtype=torch.int64, device=dev)
    _check("attn_selftest_fp8_quotients",
           lib().attn_selftest_fp8_quotients(out.data_ptr(), _stream_handle(stream, dev)))
    torch.cuda.synchronize(dev)
    return int(out.item())


def decode_status(code: int) -> dict:
    """Split a device status word into kind, role and wait site."""
    return {"kind": code & 0xFF, "role": (code >> 8) & 0xFF, "site": (code >> 16) & 0xFF}


def version() -> int:
    return int(lib().attn_version())
