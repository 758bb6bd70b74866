"""Thin ctypes binding of libh3attn (the H3 attention step on one GB300).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libh3attn.so``.  PyTorch supplies device memory and streams.
There is no CPU or eager fallback: if the library is missing or the device
is not sm_103, calls raise.

The entry points mirror the C ABI in ``include/h3attn.h``:

* ``h3attn_qk_norm_rope(q, k, wq, wk, cos, sin, rotary_dim, eps, stream)`` --
  fused Q/K RMSNorm, bf16 boundary and partial RoPE, in place (FastVideo
  PR #1832 "Add FlashInfer attention backend support for MiniMax H3",
  section "Preserve H3-specific attention behavior").
* ``h3attn_qk_norm_rope_out(q, k, q_out, k_out, ...)`` -- the same step into
  separate outputs, leaving the raw q and k in place (SGLang PR #37903
  "[diffusion] model: support VDN-H3 ...", section "Modifications": the
  out-of-place variant, bit-equal to the in-place one, keeps the raw q/k).
* ``h3attn_prefill_window(q, k, v, o, window, scale, mask, stream)`` -- the
  chunked window with anchor frames of SGLang PR #37903 ("Modifications",
  hybrid_window_attn_h3), key tiles outside a query block's window skipped.
* ``h3attn_rmsnorm_modulate(x, y, w, scale, shift, idx, eps, stream)`` --
  fused RMSNorm -> indexed AdaLN scale/shift modulation of DiT hidden rows
  with the bf16 boundaries of the unfused path (TeleFuser PR #37, section
  2.5).
* ``h3attn_prefill(q, k, v, o, scale, mask, causal, stream)`` -- dense
  prefill attention on BSHD bf16 tensors with GQA, cross-attention, causal
  and boolean-mask variants (FastVideo PR #1799 "Add opt-in FlashInfer
  attention backend for Wan", section "Implementation").

Generation over a paged key-value cache (``PagedKV``), one step of a block:

* ``h3attn_add_rmsnorm(x, residual, h, y, w, eps, y_scale, stream)`` --
  residual add and RMSNorm, in bf16 or in e4m3 with scales.
* ``h3attn_qk_norm_rope_append(q, k, v, q_out, cache, ...)`` -- the fused
  Q/K norm and RoPE of new tokens, K and V appended to the cache.
* ``h3attn_paged_decode(q, o, cache, scale, workspace, stream)`` -- attention
  of one new token per sequence over the cache.
* ``h3attn_rope_table(cos, sin, rotary_dim, theta, scaling, pos, first,
  stream)`` -- rotary tables, also scaled for long contexts.

and what keeps the cache small:

* ``h3attn_qk_norm_rope_append_q4(q, k, v, q_out, cache, ...)`` -- the append
  into a cache in 4 bits (``PagedKV4``).
* ``h3attn_paged_decode_q4(q, o, cache, scale, workspace, stream)`` -- the
  decode attention over it.
* ``h3attn_paged_read(cache, k, v, first, stream)`` -- tokens of either cache
  as contiguous rows, for a prefill that goes on from them.
* ``h3attn_paged_decode_weights(q, o, cache, weights, workspace, scale,
  stream)`` -- the decode attention of either cache, with what each token was
  attended to added up.
* ``h3attn_paged_evict(cache, weights, keep, recent, len_out, workspace,
  stream)`` -- eviction of the tokens that were attended to least.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libh3attn.so")

H3ATTN_OK = 0
H3ATTN_ERR_INVALID_ARG = 1
H3ATTN_ERR_MISALIGNED = 2
H3ATTN_ERR_UNSUPPORTED_HEAD_DIM = 3
H3ATTN_ERR_UNSUPPORTED_DEVICE = 4
H3ATTN_ERR_UNSUPPORTED_MASK = 5
H3ATTN_ERR_LAUNCH = 6
H3ATTN_ERR_TIMEOUT = 7

# Every symbol include/h3attn.h declares.
EXPORTED = ("h3attn_qk_norm_rope", "h3attn_qk_norm_rope_out", "h3attn_prefill", "h3attn_prefill_ws",
            "h3attn_prefill_workspace_size", "h3attn_prefill_noalloc", "h3attn_prefill_window",
            "h3attn_rmsnorm_modulate", "h3attn_add_rmsnorm", "h3attn_rope_table", "h3attn_qk_norm_rope_append",
            "h3attn_paged_decode", "h3attn_paged_decode_workspace_size",
            "h3attn_qk_norm_rope_append_q4", "h3attn_paged_read", "h3attn_paged_read_q4", "h3attn_paged_decode_q4",
            "h3attn_paged_decode_q4_workspace_size", "h3attn_paged_decode_weights",
            "h3attn_paged_decode_weights_workspace_size", "h3attn_paged_decode_weights_q4",
            "h3attn_paged_decode_weights_q4_workspace_size", "h3attn_paged_evict", "h3attn_paged_evict_q4",
            "h3attn_paged_evict_workspace_size",
            "h3attn_status_string", "h3attn_check_device_status", "h3attn_version")


class H3AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.h3attn_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


class h3attn_mask_t(ctypes.Structure):
    _fields_ = [("kv_len", ctypes.c_void_p), ("q_len", ctypes.c_void_p),
                ("causal_b", ctypes.c_void_p), ("bits", ctypes.c_void_p)]


class h3attn_window_t(ctypes.Structure):
    _fields_ = [("frame_tokens", ctypes.c_int), ("anchor_frames", ctypes.c_int),
                ("chunk_frames", ctypes.c_int), ("radius", ctypes.c_int)]


class h3attn_paged_kv_t(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("B", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int)]


class h3attn_paged_kv4_t(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("B", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int)]


class h3attn_rope_scaling_t(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("original_len", ctypes.c_int), ("factor", ctypes.c_double),
                ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double), ("amplitude", ctypes.c_double)]


# h3attn_y_format_t and h3attn_rope_kind_t
H3ATTN_Y_BF16, H3ATTN_Y_E4M3_ROW, H3ATTN_Y_E4M3_MX32 = 0, 1, 2
H3ATTN_ROPE_NONE, H3ATTN_ROPE_LINEAR, H3ATTN_ROPE_NTK, H3ATTN_ROPE_BY_PARTS = 0, 1, 2, 3

_lock = threading.Lock()
_lib = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libh3attn.so for sm_103a in this directory."""
    from . import _build
    return _build.build(force=force, verbose=verbose)


def load(path: str = LIB_PATH):
    """Load libh3attn.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with video_dit_dense_gb300.build()")
            lib = ctypes.CDLL(path)
            P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            lib.h3attn_qk_norm_rope.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, P]
            lib.h3attn_qk_norm_rope.restype = I
            lib.h3attn_qk_norm_rope_out.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]
            lib.h3attn_qk_norm_rope_out.restype = I
            lib.h3attn_rmsnorm_modulate.argtypes = [P, P, P, P, P, P, I, I, I, F, P]
            lib.h3attn_rmsnorm_modulate.restype = I
            lib.h3attn_prefill.argtypes = [P, P, P, P, I, I, I, I, I, I, F,
                                           ctypes.POINTER(h3attn_mask_t), I, P]
            lib.h3attn_prefill.restype = I
            lib.h3attn_prefill_ws.argtypes = [P, P, P, P, I, I, I, I, I, I, F,
                                              ctypes.POINTER(h3attn_mask_t), I, P, ctypes.c_size_t, P]
            lib.h3attn_prefill_ws.restype = I
            lib.h3attn_prefill_workspace_size.argtypes = [I, I, I, I, I, I, ctypes.POINTER(h3attn_mask_t), I,
                                                          ctypes.POINTER(ctypes.c_size_t)]
            lib.h3attn_prefill_workspace_size.restype = I
            lib.h3attn_prefill_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, I, F,
                                                   ctypes.POINTER(h3attn_mask_t), I, P]
            lib.h3attn_prefill_noalloc.restype = I
            lib.h3attn_prefill_window.argtypes = [P, P, P, P, I, I, I, I, I, F, ctypes.POINTER(h3attn_window_t),
                                                  ctypes.POINTER(h3attn_mask_t), P]
            lib.h3attn_prefill_window.restype = I
            cache = ctypes.POINTER(h3attn_paged_kv_t)
            lib.h3attn_add_rmsnorm.argtypes = [P, P, P, P, P, P, I, I, I, F, P]
            lib.h3attn_add_rmsnorm.restype = I
            lib.h3attn_rope_table.argtypes = [P, P, P, ctypes.c_int64, I, I, ctypes.c_double,
                                              ctypes.POINTER(h3attn_rope_scaling_t), P]
            lib.h3attn_rope_table.restype = I
            lib.h3attn_qk_norm_rope_append.argtypes = [P, P, P, P, cache, P, P, P, P, P, P, P, I, I, ctypes.c_int64,
                                                       ctypes.c_int64, ctypes.c_int64, I, I, I, F, P]
            lib.h3attn_qk_norm_rope_append.restype = I
            lib.h3attn_paged_decode.argtypes = [P, P, cache, I, F, P, ctypes.c_size_t, P]
            lib.h3attn_paged_decode.restype = I
            lib.h3attn_paged_decode_workspace_size.argtypes = [cache, I, ctypes.POINTER(ctypes.c_size_t)]
            lib.h3attn_paged_decode_workspace_size.restype = I
            cache4, sized = ctypes.POINTER(h3attn_paged_kv4_t), ctypes.POINTER(ctypes.c_size_t)
            lib.h3attn_qk_norm_rope_append_q4.argtypes = [cache4 if t is cache else t
                                                          for t in lib.h3attn_qk_norm_rope_append.argtypes]
            lib.h3attn_paged_decode_q4.argtypes = [P, P, cache4, I, F, P, ctypes.c_size_t, P]
            lib.h3attn_paged_decode_q4_workspace_size.argtypes = [cache4, I, sized]
            for c, suffix in ((cache, ""), (cache4, "_q4")):
                getattr(lib, "h3attn_paged_read" + suffix).argtypes = [c, P, P, P, I, P]
                getattr(lib, "h3attn_paged_decode_weights" + suffix).argtypes = [P, P, c, I, F, P, P, ctypes.c_size_t, P]
                getattr(lib, f"h3attn_paged_decode_weights{suffix}_workspace_size").argtypes = [c, I, sized]
                getattr(lib, "h3attn_paged_evict" + suffix).argtypes = [c, P, I, I, P, P, ctypes.c_size_t, P]
            lib.h3attn_paged_evict_workspace_size.argtypes = [I, I, I, I, I, sized]
            for name in EXPORTED:
                getattr(lib, name).restype = I
            lib.h3attn_status_string.argtypes = [I]
            lib.h3attn_status_string.restype = ctypes.c_char_p
            lib.h3attn_check_device_status.argtypes = [P]
            lib.h3attn_check_device_status.restype = I
            lib.h3attn_version.argtypes = []
            lib.h3attn_version.restype = I
            _lib = lib
    return _lib


def lib():
    return load()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_bf16(name, t):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous 4-D bf16 CUDA tensor (BSHD)")
    if t.requires_grad:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name}: inference only, grad-enabled inputs are rejected")


def _raise_if(status, where):
    if status != H3ATTN_OK:
        raise H3AttnError(status, where)


def _norm_rope_args(q, k, wq, wk, cos, sin, rotary_dim):
    if q is None and k is None:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "at least one of q and k must be given")
    ref = q if q is not None else k
    if q is not None:
        _check_bf16("q", q)
    if k is not None:
        _check_bf16("k", k)
    B, S, _, D = ref.shape
    Hq = q.shape[2] if q is not None else 0
    Hkv = k.shape[2] if k is not None else 0
    if k is not None and q is not None and (k.shape[0], k.shape[1], k.shape[3]) != (B, S, D):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "q and k must share batch, sequence and head_dim")
    import torch
    for name, t in (("wq", wq), ("wk", wk), ("cos", cos), ("sin", sin)):
        if t is not None and (t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous()):
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous float32 CUDA tensor")
    # the kernel reads D weights per row: a shorter tensor would be read past its end
    for name, rows, w in (("wq", q, wq), ("wk", k, wk)):
        if rows is not None and (w is None or w.numel() != D):
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be a [{D}] float32 CUDA tensor")
    if rotary_dim > 0:
        if cos is None or sin is None:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "cos and sin are required when rotary_dim > 0")
        if cos.shape[-1] != rotary_dim // 2 or cos.numel() < S * (rotary_dim // 2) or sin.shape != cos.shape:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "cos/sin must be [>=S, rotary_dim/2]")
    return B, S, Hq, Hkv, D


def h3attn_qk_norm_rope(q, k, wq, wk, cos, sin, rotary_dim=96, eps=1e-6, stream=None):
    """In-place fused Q/K RMSNorm + bf16 boundary + partial RoPE.

    q: [B, S, Hq, D] bf16, k: [B, S, Hkv, D] bf16 (either may be None);
    wq, wk: [D] float32; cos, sin: [>=S, rotary_dim/2] float32.
    """
    load()
    B, S, Hq, Hkv, D = _norm_rope_args(q, k, wq, wk, cos, sin, rotary_dim)
    st = _lib.h3attn_qk_norm_rope(_ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(cos), _ptr(sin),
                                  B, S, Hq, Hkv, D, int(rotary_dim), float(eps), _stream_handle(stream))
    _raise_if(st, "h3attn_qk_norm_rope")


def h3attn_qk_norm_rope_out(q, k, q_out, k_out, wq, wk, cos, sin, rotary_dim=96, eps=1e-6, stream=None):
    """Out-of-place fused Q/K RMSNorm + bf16 boundary + partial RoPE: q and k
    are read only; q_out, k_out (same shapes, preallocated) receive the
    result, bit-identical to the in-place call."""
    load()
    B, S, Hq, Hkv, D = _norm_rope_args(q, k, wq, wk, cos, sin, rotary_dim)
    for name, src, dst in (("q_out", q, q_out), ("k_out", k, k_out)):
        if (src is None) != (dst is None):
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be given exactly when its input is")
        if dst is not None:
            _check_bf16(name, dst)
            if tuple(dst.shape) != tuple(src.shape):
                raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must have the shape of its input")
    st = _lib.h3attn_qk_norm_rope_out(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(wq), _ptr(wk), _ptr(cos),
                                      _ptr(sin), B, S, Hq, Hkv, D, int(rotary_dim), float(eps),
                                      _stream_handle(stream))
    _raise_if(st, "h3attn_qk_norm_rope_out")
    return q_out, k_out


@dataclass
class Mask:
    """Mask descriptor (device tensors, per batch item): see h3attn_mask_t."""
    kv_len: object = None    # int32 [B]
    q_len: object = None     # int32 [B]
    causal_b: object = None  # uint8 [B]
    bits: object = None      # int32/uint32 [B, Sq, ceil(Sk/32)]


def _mask_struct(mask: Mask, B: int):
    """Checks the per-sample fields of a mask and packs its pointers into an
    h3attn_mask_t (the kernels read B entries of each field given)."""
    import torch
    for name, t, dt in (("kv_len", mask.kv_len, torch.int32), ("q_len", mask.q_len, torch.int32),
                        ("causal_b", mask.causal_b, torch.uint8)):
        if t is not None and (t.dtype != dt or t.numel() != B or not t.is_cuda or not t.is_contiguous()):
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous [{B}] {dt} CUDA tensor")
    return ctypes.pointer(h3attn_mask_t(_ptr(mask.kv_len), _ptr(mask.q_len), _ptr(mask.causal_b), _ptr(mask.bits)))


def h3attn_prefill(q, k, v, o, scale=None, mask: Mask | None = None, causal=False, stream=None, workspace=None):
    """o <- softmax(q k^T * scale) v on BSHD bf16 tensors (o preallocated).

    workspace: None, or a CUDA tensor of at least h3attn_prefill_workspace_size()
    bytes for the split-key tail (the call then goes through h3attn_prefill_ws).
    """
    load()
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check_bf16(name, t)
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape) or tuple(o.shape) != tuple(q.shape):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "shape mismatch between q, k, v and o")
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    mptr = None
    if mask is not None:
        if mask.bits is not None:
            if mask.bits.dim() == 4:
                raise H3AttnError(H3ATTN_ERR_UNSUPPORTED_MASK, "per-head [B, H, Q, K] masks are not supported")
            W = (Sk + 31) // 32
            if tuple(mask.bits.shape) != (B, Sq, W) or mask.bits.element_size() != 4 or \
                    not mask.bits.is_cuda or not mask.bits.is_contiguous():
                raise H3AttnError(H3ATTN_ERR_INVALID_ARG,
                                  f"bits must be contiguous 32-bit CUDA words of shape [{B}, {Sq}, {W}]")
        mptr = _mask_struct(mask, B)
    if workspace is None:
        st = _lib.h3attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Sq, Sk, Hq, Hkv, D, float(scale), mptr,
                                 int(bool(causal)), _stream_handle(stream))
        _raise_if(st, "h3attn_prefill")
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "workspace must be a contiguous CUDA tensor")
        nbytes = workspace.numel() * workspace.element_size()
        st = _lib.h3attn_prefill_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Sq, Sk, Hq, Hkv, D, float(scale), mptr,
                                    int(bool(causal)), _ptr(workspace), nbytes, _stream_handle(stream))
        _raise_if(st, "h3attn_prefill_ws")
    return o


def h3attn_prefill_workspace_size(B, Sq, Sk, Hq, Hkv, D, mask: Mask | None = None, causal=False) -> int:
    """Bytes of workspace the split-key tail needs for this call (0: no split).
    Only the presence of the mask fields matters, not their values."""
    load()
    mptr = None
    if mask is not None:
        mptr = ctypes.pointer(h3attn_mask_t(_ptr(mask.kv_len), _ptr(mask.q_len), _ptr(mask.causal_b),
                                            _ptr(mask.bits)))
    out = ctypes.c_size_t(0)
    st = _lib.h3attn_prefill_workspace_size(B, Sq, Sk, Hq, Hkv, D, mptr, int(bool(causal)), ctypes.byref(out))
    _raise_if(st, "h3attn_prefill_workspace_size")
    return int(out.value)


# Bytes of the fixed scratch array behind h3attn_prefill_noalloc.
NOALLOC_SCRATCH_BYTES = 12 << 20


def h3attn_prefill_noalloc(q, k, v, o, scale=None, mask: Mask | None = None, causal=False, stream=None):
    """h3attn_prefill with the split-key tail's scratch in the library's fixed
    12 MiB device array: the call allocates nothing (for hosts that cannot
    allocate device memory).  Calls whose kernels may overlap must be ordered
    by the caller, since they share the array."""
    load()
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check_bf16(name, t)
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape) or tuple(o.shape) != tuple(q.shape):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "shape mismatch between q, k, v and o")
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    mptr = None if mask is None else _mask_struct(mask, B)
    need = h3attn_prefill_workspace_size(B, Sq, Sk, Hq, Hkv, D, mask, causal)
    if need > NOALLOC_SCRATCH_BYTES:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"h3attn_prefill_noalloc: this call needs {need} bytes of "
                                                  f"scratch, more than the fixed {NOALLOC_SCRATCH_BYTES}")
    st = _lib.h3attn_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Sq, Sk, Hq, Hkv, D, float(scale), mptr,
                                     int(bool(causal)), _stream_handle(stream))
    _raise_if(st, "h3attn_prefill_noalloc")
    return o


def prefill_workspace(q, k, mask: Mask | None = None, causal=False):
    """A workspace tensor sized for prefill(q, k, ...) on the current device,
    or None when the call would not split (allocated by torch: the library
    allocates nothing)."""
    import torch
    B, Sq, Hq, D = q.shape
    n = h3attn_prefill_workspace_size(B, Sq, k.shape[1], Hq, k.shape[2], D, mask, causal)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def h3attn_rmsnorm_modulate(x, y, w, scale, shift, idx=None, eps=1e-6, stream=None):
    """y <- bf16(bf16(bf16(rmsnorm(x) * w) * bf16(1 + scale[idx])) + shift[idx]) row by row.

    x, y: [T, C] bf16 CUDA tensors (y may be x); w: [C] float32 or None;
    scale, shift: [N, C] bf16; idx: [T] int32 or None (table row 0 for all).
    """
    import torch
    load()
    for name, t in (("x", x), ("y", y), ("scale", scale), ("shift", shift)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous 2-D bf16 CUDA tensor")
    T, C = x.shape
    N = scale.shape[0]
    if tuple(y.shape) != (T, C) or tuple(scale.shape) != (N, C) or tuple(shift.shape) != (N, C):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "shape mismatch between x, y, scale and shift")
    if w is not None and (w.dtype != torch.float32 or not w.is_cuda or w.numel() != C):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"w must be a [{C}] float32 CUDA tensor")
    if idx is not None and (idx.dtype != torch.int32 or not idx.is_cuda or idx.numel() != T):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"idx must be a [{T}] int32 CUDA tensor")
    st = _lib.h3attn_rmsnorm_modulate(_ptr(x), _ptr(y), _ptr(w), _ptr(scale), _ptr(shift), _ptr(idx), T, C, N,
                                      float(eps), _stream_handle(stream))
    _raise_if(st, "h3attn_rmsnorm_modulate")
    return y


@dataclass
class Window:
    """Chunked window with anchor frames: see h3attn_window_t."""
    frame_tokens: int
    anchor_frames: int
    chunk_frames: int
    radius: int


def h3attn_prefill_window(q, k, v, o, window: Window, scale=None, mask: Mask | None = None, stream=None):
    """o <- windowed self-attention of q against k, v (BSHD bf16, Sq == Sk)."""
    load()
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check_bf16(name, t)
    B, S, Hq, D = q.shape
    if tuple(k.shape[:2]) != (B, S) or k.shape[3] != D or tuple(v.shape) != tuple(k.shape) or \
            tuple(o.shape) != tuple(q.shape):
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "shape mismatch between q, k, v and o (self-attention)")
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    mptr = None
    if mask is not None:
        if mask.bits is not None or mask.causal_b is not None:
            raise H3AttnError(H3ATTN_ERR_UNSUPPORTED_MASK, "the window combines with kv_len / q_len only")
        mptr = _mask_struct(mask, B)
    w = h3attn_window_t(int(window.frame_tokens), int(window.anchor_frames), int(window.chunk_frames),
                        int(window.radius))
    st = _lib.h3attn_prefill_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, S, Hq, k.shape[2], D, float(scale),
                                    ctypes.pointer(w), mptr, _stream_handle(stream))
    _raise_if(st, "h3attn_prefill_window")
    return o


# The generation operators are called for every token, where a call's kernels
# take a few microseconds: their argument checks and the call itself are compiled
# (csrc/step.cpp, _step.so), the functions here give them their names.
_bound = None


def _get_step():
    """The compiled host path, given the loaded library's entry points."""
    global _bound
    if _bound is None:
        lib = load()
        import torch  # the module is linked against torch's libraries
        from . import _build
        if not os.path.exists(_build.STEP_LIB):
            raise RuntimeError("_step.so is missing: build it with video_dit_dense_gb300.build()")
        built_for, running = _build.step_built_for(), _build.step_versions(torch)
        if built_for != running:  # before it is loaded: another version's layouts would be read
            raise RuntimeError(f"_step.so was built for {built_for or 'versions that are not known'}, this is {running}: "
                               "build it with video_dit_dense_gb300.build()")
        module = importlib.import_module("._step", __name__)
        module.bind(H3AttnError, PagedKV, PagedKV4, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.h3attn_add_rmsnorm, lib.h3attn_rope_table, lib.h3attn_qk_norm_rope_append, lib.h3attn_paged_decode,
            lib.h3attn_qk_norm_rope_append_q4, lib.h3attn_paged_decode_q4, lib.h3attn_paged_decode_weights,
            lib.h3attn_paged_decode_weights_q4, lib.h3attn_paged_read, lib.h3attn_paged_read_q4, lib.h3attn_paged_evict,
            lib.h3attn_paged_evict_q4)))
        _bound = module
    return _bound


def h3attn_add_rmsnorm(x, residual, h, y, w=None, eps=1e-6, y_scale=None, stream=None):
    """h <- bf16(x + residual); y <- rmsnorm(h) * w, in bf16 or in e4m3 with scales.

    x, residual, h: [T, C] bf16 CUDA tensors (residual and h may both be None:
    the norm is then of x; h may be x or residual); w: [C] float32 or None.
    y: [T, C], bfloat16, or float8_e4m3fn with y_scale [T] float32 (one scale a
    row) or [T, C / 32] float8_e8m0fnu or uint8 (a power of two for each 32
    channels, row by row).  Returns y.
    """
    return (_bound or _get_step()).add_rmsnorm(x, residual, h, y, w, eps, y_scale, stream)


_ROPE_KINDS = {"none": H3ATTN_ROPE_NONE, "linear": H3ATTN_ROPE_LINEAR, "ntk": H3ATTN_ROPE_NTK,
               "by_parts": H3ATTN_ROPE_BY_PARTS}


@dataclass(frozen=True)
class RopeScaling:
    """Rotary frequencies for long contexts: see h3attn_rope_scaling_t.  kind
    is "none", "linear", "ntk" or "by_parts"."""
    kind: str
    factor: float = 1.0
    original_len: int = 1
    low_turns: float = 1.0
    high_turns: float = 32.0
    amplitude: float = 1.0

    def __post_init__(self):
        if self.kind not in _ROPE_KINDS:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"unknown scaling {self.kind!r}")
        if not -2 ** 31 <= self.original_len < 2 ** 31:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "original_len must fit 32 bits")
        object.__setattr__(self, "_struct", h3attn_rope_scaling_t(_ROPE_KINDS[self.kind], self.original_len, self.factor,
                                                                  self.low_turns, self.high_turns, self.amplitude))


def h3attn_rope_table(cos, sin, rotary_dim, theta=10000.0, scaling: RopeScaling | None = None, pos=None, first=0,
                      stream=None):
    """cos, sin <- the rotary table of positions pos, or first, first + 1, ...

    cos, sin: [N, rotary_dim / 2] float32 CUDA tensors (preallocated); pos: [N]
    int32 or None.  Returns (cos, sin).
    """
    (_bound or _get_step()).rope_table(cos, sin, rotary_dim, theta,
                                      0 if scaling is None else ctypes.addressof(scaling._struct), pos, first, stream)
    return cos, sin


def _check(name, t, dtype, shape, dev):
    """A contiguous tensor of this dtype and shape on CUDA device dev, without a
    gradient."""
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != shape:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous {list(shape)} {dtype} CUDA tensor")
    if t.requires_grad:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name}: inference only, grad-enabled inputs are rejected")
    if t.get_device() != dev:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must be on the cache's device")


class PagedKV:
    """A paged key-value cache: see h3attn_paged_kv_t.

    k_pages, v_pages: [num_pages, page_size, Hkv, D] bf16; page_table:
    [B, max_pages] int32; kv_len: [B] int32, the tokens the cache holds of each
    sequence.  All CUDA tensors on one device, kept by reference: their
    contents may change between calls, their storage not.
    """
    __slots__ = ("_tensors", "_struct", "_address", "_device")

    def __init__(self, k_pages, v_pages, page_table, kv_len):
        import torch
        if k_pages.dim() != 4 or page_table.dim() != 2:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "pages must be [num_pages, page_size, Hkv, D], page_table [B, max_pages]")
        num_pages, page_size, Hkv, D = k_pages.shape
        B, max_pages = page_table.shape
        if max(num_pages, page_size, Hkv, D, B, max_pages) >= 2 ** 31:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "the cache's sizes must fit 32 bits")
        self._device = k_pages.get_device()
        _check("k_pages", k_pages, torch.bfloat16, (num_pages, page_size, Hkv, D), self._device)
        _check("v_pages", v_pages, torch.bfloat16, (num_pages, page_size, Hkv, D), self._device)
        _check("page_table", page_table, torch.int32, (B, max_pages), self._device)
        _check("kv_len", kv_len, torch.int32, (B,), self._device)
        self._tensors = (k_pages, v_pages, page_table, kv_len)
        self._struct = h3attn_paged_kv_t(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                                         kv_len.data_ptr(), B, num_pages, page_size, max_pages, Hkv, D)
        self._address = ctypes.addressof(self._struct)

    k_pages = property(lambda self: self._tensors[0])
    v_pages = property(lambda self: self._tensors[1])
    page_table = property(lambda self: self._tensors[2])
    kv_len = property(lambda self: self._tensors[3])

    def with_lengths(self, kv_len):
        """The same cache with another lengths tensor (len_out of an append)."""
        return PagedKV(self.k_pages, self.v_pages, self.page_table, kv_len)


class PagedKV4:
    """A paged key-value cache in 4 bits: see h3attn_paged_kv4_t.

    k_codes, v_codes: [num_pages, page_size, Hkv, D / 2] uint8; k_scales,
    v_scales: [num_pages, page_size, Hkv, D / 16] uint8; page_table and kv_len as
    in PagedKV.  Kept by reference like there.
    """
    __slots__ = ("_tensors", "_struct", "_address", "_device")

    def __init__(self, k_codes, v_codes, k_scales, v_scales, page_table, kv_len):
        import torch
        if k_codes.dim() != 4 or page_table.dim() != 2:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG,
                              "codes must be [num_pages, page_size, Hkv, D / 2], page_table [B, max_pages]")
        num_pages, page_size, Hkv, half = k_codes.shape
        B, max_pages = page_table.shape
        D = 2 * half
        if max(num_pages, page_size, Hkv, D, B, max_pages) >= 2 ** 31:
            raise H3AttnError(H3ATTN_ERR_INVALID_ARG, "the cache's sizes must fit 32 bits")
        self._device = k_codes.get_device()
        for name, t, n in (("k_codes", k_codes, 2), ("v_codes", v_codes, 2), ("k_scales", k_scales, 16), ("v_scales", v_scales, 16)):
            _check(name, t, torch.uint8, (num_pages, page_size, Hkv, D // n), self._device)
        _check("page_table", page_table, torch.int32, (B, max_pages), self._device)
        _check("kv_len", kv_len, torch.int32, (B,), self._device)
        self._tensors = (k_codes, v_codes, k_scales, v_scales, page_table, kv_len)
        self._struct = h3attn_paged_kv4_t(*(t.data_ptr() for t in self._tensors), B, num_pages, page_size, max_pages, Hkv, D)
        self._address = ctypes.addressof(self._struct)

    k_codes = property(lambda self: self._tensors[0])
    v_codes = property(lambda self: self._tensors[1])
    k_scales = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])
    page_table = property(lambda self: self._tensors[4])
    kv_len = property(lambda self: self._tensors[5])

    def with_lengths(self, kv_len):
        """The same cache with another lengths tensor (len_out of an append or an eviction)."""
        return PagedKV4(*self._tensors[:5], kv_len)


def h3attn_qk_norm_rope_append(q, k, v, q_out, cache: PagedKV, wq, wk, cos, sin, rotary_dim=96, eps=1e-6,
                               interleaved=False, pos=None, new_len=None, len_out=None, stream=None):
    """Q/K RMSNorm + bf16 boundary + partial RoPE of new tokens; K and V go to
    the cache behind its kv_len tokens, Q to q_out.

    q: [B, S, Hq, D] bf16 or None, k, v: [B, S, Hkv, D] bf16 (slices of one
    projection are taken as they are); q_out: contiguous [B, S, Hq, D], or None
    with q; wq, wk: [D] float32 or None (no norm); cos, sin: [rows,
    rotary_dim / 2] float32; pos: [B, S] int32 or None (the place in the cache);
    new_len: [B] int32 or None (all S); len_out: [B] int32 or None, receives the
    new lengths.  Returns q_out.
    """
    return (_bound or _get_step()).append(q, k, v, q_out, cache, wq, wk, cos, sin, rotary_dim, eps, interleaved, pos, new_len,
                                         len_out, stream)


def h3attn_paged_decode(q, o, cache: PagedKV, scale=None, workspace=None, stream=None):
    """o <- attention of one new token per sequence over its paged cache.

    q, o: [B, 1, Hq, D] or [B, Hq, D] bf16 (o preallocated); the token's own key
    and value are in the cache.  workspace: None (one CTA walks a sequence), or
    a CUDA tensor from paged_decode_workspace(): the sequences, up to 512, are
    then split over the GPU.  Returns o.
    """
    return (_bound or _get_step()).decode(q, o, cache, scale, workspace, stream)


def h3attn_paged_decode_workspace_size(cache: PagedKV, Hq) -> int:
    """Bytes of workspace h3attn_paged_decode takes for this cache and Hq query heads (0: no split)."""
    return _sized("h3attn_paged_decode_workspace_size", ctypes.byref(cache._struct), _int32("Hq", Hq))


def paged_decode_workspace(q, cache: PagedKV):
    """A workspace tensor for h3attn_paged_decode(q, ..., cache) on the current
    device, or None when the call does not split (allocated by torch)."""
    n = h3attn_paged_decode_workspace_size(cache, q.shape[-2])
    import torch
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def h3attn_qk_norm_rope_append_q4(q, k, v, q_out, cache: PagedKV4, wq, wk, cos, sin, rotary_dim=96, eps=1e-6,
                                  interleaved=False, pos=None, new_len=None, len_out=None, stream=None):
    """h3attn_qk_norm_rope_append into a cache in 4 bits: the same arguments, the
    same q_out and len_out; K and V rows are stored as codes and scales."""
    return (_bound or _get_step()).append_q4(q, k, v, q_out, cache, wq, wk, cos, sin, rotary_dim, eps, interleaved, pos, new_len,
                                            len_out, stream)


def h3attn_paged_read(cache, k, v, first=None, stream=None):
    """k, v <- the tokens first[b], first[b] + 1, ... of each sequence.

    cache: a PagedKV or a PagedKV4; k, v: contiguous [B, S, Hkv, D] bf16 (either
    may be None); first: [B] int32 or None (from token 0).  Rows of tokens that
    the cache does not hold are left as they are.  Returns (k, v).
    """
    (_bound or _get_step()).read(cache, k, v, first, stream)
    return k, v


def h3attn_paged_decode_q4(q, o, cache: PagedKV4, scale=None, workspace=None, stream=None):
    """h3attn_paged_decode over a cache in 4 bits; workspace: None, or a CUDA
    tensor from paged_decode_q4_workspace().  Returns o."""
    return (_bound or _get_step()).decode_q4(q, o, cache, scale, workspace, stream)


def h3attn_paged_decode_weights(q, o, cache, weights, workspace, scale=None, stream=None):
    """The decode attention of a PagedKV or a PagedKV4, with each token's
    attention weights, summed over the query heads, added to weights: [B,
    max_pages * page_size] float32.  workspace: a CUDA tensor from
    paged_decode_weights_workspace().  Returns o.
    """
    return (_bound or _get_step()).decode_weights(q, o, cache, scale, weights, workspace, stream)


def h3attn_paged_evict(cache, weights, keep, recent, len_out, workspace, stream=None):
    """Brings each sequence of more than keep tokens back to keep: its recent
    last ones, and of the others the heaviest by weights.

    cache: a PagedKV or a PagedKV4, whose rows move; weights: [B, max_pages *
    page_size] float32, moved with them; len_out: [B] int32, the lengths after it
    (for cache.with_lengths); workspace: a CUDA tensor from
    paged_evict_workspace().  Returns len_out.
    """
    return (_bound or _get_step()).evict(cache, weights, keep, recent, len_out, workspace, stream)


def _int32(name, n) -> int:
    """n for the C interface: ctypes would take it modulo 2^32."""
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise H3AttnError(H3ATTN_ERR_INVALID_ARG, f"{name} must fit 32 bits")
    return n


def _sized(entry, *args) -> int:
    out = ctypes.c_size_t(0)
    _raise_if(getattr(load(), entry)(*args, ctypes.byref(out)), entry)
    return int(out.value)


def _workspace(n, device):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def h3attn_paged_decode_q4_workspace_size(cache: PagedKV4, Hq) -> int:
    """Bytes of workspace h3attn_paged_decode_q4 takes for this cache and Hq query heads (0: no split)."""
    return _sized("h3attn_paged_decode_q4_workspace_size", ctypes.byref(cache._struct), _int32("Hq", Hq))


def paged_decode_q4_workspace(q, cache: PagedKV4):
    """A workspace tensor for h3attn_paged_decode_q4(q, ..., cache) on the current
    device, or None when the call does not split (allocated by torch)."""
    return _workspace(h3attn_paged_decode_q4_workspace_size(cache, q.shape[-2]), q.device)


def h3attn_paged_decode_weights_workspace_size(cache, Hq) -> int:
    """Bytes of workspace h3attn_paged_decode_weights takes for this cache (of either kind) and Hq query heads."""
    kind = "_q4" if isinstance(cache, PagedKV4) else ""
    return _sized(f"h3attn_paged_decode_weights{kind}_workspace_size", ctypes.byref(cache._struct), _int32("Hq", Hq))


def paged_decode_weights_workspace(q, cache):
    """A workspace tensor for h3attn_paged_decode_weights(q, ..., cache) on the
    current device (allocated by torch; None for an empty batch)."""
    return _workspace(h3attn_paged_decode_weights_workspace_size(cache, q.shape[-2]), q.device)


def h3attn_paged_evict_workspace_size(cache, keep, recent) -> int:
    """Bytes of workspace h3attn_paged_evict takes for this cache (of either kind), keep and recent."""
    s = cache._struct
    return _sized("h3attn_paged_evict_workspace_size", s.B, s.page_size, s.max_pages, _int32("keep", keep), _int32("recent", recent))


def paged_evict_workspace(cache, keep, recent):
    """A workspace tensor for h3attn_paged_evict(cache, ..., keep, recent)
    (allocated by torch on the cache's device; None for an empty batch)."""
    return _workspace(h3attn_paged_evict_workspace_size(cache, keep, recent), cache.page_table.device)


def h3attn_check_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    load()
    return _lib.h3attn_check_device_status(_stream_handle(stream))


def h3attn_status_string(status: int) -> str:
    return load().h3attn_status_string(status).decode()


def h3attn_version() -> int:
    return load().h3attn_version()


# Short aliases.
qk_norm_rope = h3attn_qk_norm_rope
prefill = h3attn_prefill
check_device_status = h3attn_check_device_status
