"""Python binding of the C ABI declared in ``include/attn.h``.

Argument marshalling only: every step of the attention runs in the CUDA
library ``libattn.so`` (the calls of a decode step reach it through the native
module ``_binding``, the others through ctypes). There is no fallback of any kind; if the library has
not been built, or the device is not an sm_103 GPU, the calls fail loudly.

``attn_fwd`` and the other functions keep the C names and take raw device
pointers (ints); ``attention`` is the torch convenience wrapper that derives
the sizes from (B, S, H, D) tensors, allocates the outputs with PyTorch and
raises ``AttnError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

from . import build as _build

MASK_NONE, MASK_CAUSAL, MASK_ADDITIVE, MASK_CAUSAL_ADDITIVE = 0, 1, 2, 3
ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_DEVICE_TIMEOUT = 0, 1, 2, 3, 4
ATTN_ERR_BAD_INDEX = 5
CACHE_16BIT, CACHE_E4M3 = 0, 1

_lib = None


class AttnError(RuntimeError):
    def __init__(self, code: int, what: str = "attn_fwd"):
        self.code = code
        super().__init__(f"{what} failed: {attn_status_string(code)} ({code})")


def library_path() -> str:
    return _build.LIBRARY


def lib() -> ctypes.CDLL:
    """Load libattn.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(path)
    P, I = ctypes.c_void_p, ctypes.c_int
    for f in (L.attn_fwd, L.attn_fwd_f16):
        f.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, P, P]
        f.restype = I
    for f in (L.attn_fwd_splitkv, L.attn_fwd_splitkv_f16):
        f.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, P, I, P, ctypes.c_size_t, P]
        f.restype = I
    for f in (L.attn_fwd_rope, L.attn_fwd_rope_f16):
        f.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, P, P, I, I, I, P, I, P,
                      ctypes.c_size_t, P]
        f.restype = I
    for f in (L.attn_rope_apply, L.attn_rope_apply_f16):
        f.argtypes = [P, P, I, I, I, I, P, I, I, P]
        f.restype = I
    for f in (L.attn_fwd_host, L.attn_fwd_host_f16):
        f.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, P, P, ctypes.c_size_t, P]
        f.restype = I
    L.attn_fwd_host_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    L.attn_fwd_host_workspace_bytes.restype = ctypes.c_size_t
    L.attn_linear.argtypes = [P, P, P, P, P, I, I, I, P]
    L.attn_linear.restype = I
    L.attn_layernorm.argtypes = [P, P, P, P, I, I, ctypes.c_float, P]
    L.attn_layernorm.restype = I
    L.attn_fwd_qkvpacked.argtypes = [P, P, P, I, I, I, I, I, ctypes.c_float, I, P, P]
    L.attn_fwd_qkvpacked.restype = I
    L.attn_block_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, ctypes.c_float, I, P, ctypes.c_size_t, P]
    L.attn_block_fwd.restype = I
    L.attn_block_workspace_bytes.argtypes = [I, I, I, I, I]
    L.attn_block_workspace_bytes.restype = ctypes.c_size_t
    L.attn_rope_table.argtypes = [P, I, I, ctypes.c_double, P]
    L.attn_rope_table.restype = I
    L.attn_fwd_splitkv_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, P, I, P]
    L.attn_fwd_splitkv_noalloc.restype = I
    L.attn_splitkv_num_splits.argtypes = [I, I, I, I, I, I]
    L.attn_splitkv_num_splits.restype = I
    L.attn_splitkv_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    L.attn_splitkv_workspace_bytes.restype = ctypes.c_size_t
    for f in (L.attn_fwd_window, L.attn_fwd_window_f16):
        f.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, I, P]
        f.restype = I
    LL, F = ctypes.c_longlong, ctypes.c_float
    for f in (L.attn_kv_append, L.attn_kv_append_f16):
        f.argtypes = [P, P, LL, LL, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, I, P]
        f.restype = I
    for f in (L.attn_fwd_paged, L.attn_fwd_paged_f16):
        f.argtypes = [P, LL, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, I, P, I, P, ctypes.c_size_t, P]
        f.restype = I
    L.attn_paged_workspace_bytes.argtypes = [I, I, I, I, I, LL]
    L.attn_paged_workspace_bytes.restype = ctypes.c_size_t
    for f in (L.attn_bwd, L.attn_bwd_f16):
        f.argtypes = [P] * 9 + [LL] * 6 + [I] * 6 + [F, I, P, I, I, P, ctypes.c_size_t, P]
        f.restype = I
    L.attn_bwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    L.attn_bwd_workspace_bytes.restype = ctypes.c_size_t
    for f in (L.attn_rope_axes, L.attn_rope_axes_f16):
        f.argtypes = [P, P, LL, LL] * 2 + [I] * 5 + [P, I, P, P, I, I, P]
        f.restype = I
    L.attn_rope_axes_table.argtypes = [P, I, P, I, ctypes.c_double, P]
    L.attn_rope_axes_table.restype = I
    for f in (L.attn_checkpoint_store, L.attn_checkpoint_store_f16):
        f.argtypes = [P, LL, P, P, I, I, I, I, P]
        f.restype = I
    for f in (L.attn_checkpoint_load, L.attn_checkpoint_load_f16):
        f.argtypes = [P, P, P, LL, I, I, I, I, P]
        f.restype = I
    for f in (L.attn_bwd_checkpoint, L.attn_bwd_checkpoint_f16):
        f.argtypes = [P] * 10 + [LL] * 3 + [I] * 6 + [F, I, P, I, I, P, ctypes.c_size_t, P]
        f.restype = I
    L.attn_bwd_checkpoint_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    L.attn_bwd_checkpoint_workspace_bytes.restype = ctypes.c_size_t
    L.attn_last_status.argtypes = [P]
    L.attn_last_status.restype = I
    L.attn_status_string.argtypes = [I]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_set_wait_timeout_ns.argtypes = [ctypes.c_ulonglong]
    L.attn_set_wait_timeout_ns.restype = I
    L.attn_debug_inject_stall.argtypes = [I]
    L.attn_debug_inject_stall.restype = I
    L.attn_abi_version.argtypes = []
    L.attn_abi_version.restype = I
    _lib = L
    return L


# ---------------------------------------------------------------- raw ABI

def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, stream) -> int:
    return lib().attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, stream)


def attn_fwd_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, stream) -> int:
    return lib().attn_fwd_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, stream)


def attn_fwd_splitkv(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, num_splits,
                     workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd_splitkv(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, num_splits,
                                  workspace, workspace_bytes, stream)


def attn_fwd_splitkv_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, num_splits,
                         workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd_splitkv_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, num_splits,
                                      workspace, workspace_bytes, stream)


def attn_fwd_splitkv_noalloc(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, num_splits,
                             stream) -> int:
    """The allocation-free split-key entry point (bf16): its scratch is the library's fixed 32 MiB array."""
    return lib().attn_fwd_splitkv_noalloc(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask,
                                          num_splits, stream)


def attn_fwd_rope(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, rope_table, max_pos, q_pos0,
                  k_pos0, k_rot, num_splits, workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd_rope(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, rope_table, max_pos,
                               q_pos0, k_pos0, k_rot, num_splits, workspace, workspace_bytes, stream)


def attn_fwd_rope_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, rope_table, max_pos, q_pos0,
                      k_pos0, k_rot, num_splits, workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd_rope_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, rope_table,
                                   max_pos, q_pos0, k_pos0, k_rot, num_splits, workspace, workspace_bytes, stream)


def attn_rope_table(table, max_pos, D, base, stream) -> int:
    return lib().attn_rope_table(table, max_pos, D, float(base), stream)


def attn_rope_apply(x, y, B, S, H, D, rope_table, max_pos, pos0, stream) -> int:
    return lib().attn_rope_apply(x, y, B, S, H, D, rope_table, max_pos, pos0, stream)


def attn_rope_apply_f16(x, y, B, S, H, D, rope_table, max_pos, pos0, stream) -> int:
    return lib().attn_rope_apply_f16(x, y, B, S, H, D, rope_table, max_pos, pos0, stream)


def attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, workspace, workspace_bytes,
                  stream) -> int:
    return lib().attn_fwd_host(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, workspace,
                               workspace_bytes, stream)


def attn_fwd_host_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, workspace, workspace_bytes,
                      stream) -> int:
    return lib().attn_fwd_host_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, workspace,
                                   workspace_bytes, stream)


def attn_fwd_host_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, mask_kind) -> int:
    return int(lib().attn_fwd_host_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, mask_kind))


def attn_linear(a, w, bias, residual, out, M, N, K, stream) -> int:
    return lib().attn_linear(a, w, bias, residual, out, M, N, K, stream)


def attn_layernorm(x, gamma, beta, y, M, H, eps, stream) -> int:
    return lib().attn_layernorm(x, gamma, beta, y, M, H, eps, stream)


def attn_fwd_qkvpacked(qkv, o, lse, B, S, Hq, Hkv, D, scale, mask_kind, mask, stream) -> int:
    return lib().attn_fwd_qkvpacked(qkv, o, lse, B, S, Hq, Hkv, D, scale, mask_kind, mask, stream)


def attn_block_fwd(x, ln_gamma, ln_beta, w_qkv, b_qkv, w_o, b_o, y, B, S, Hq, Hkv, D, eps, causal, workspace,
                   workspace_bytes, stream) -> int:
    return lib().attn_block_fwd(x, ln_gamma, ln_beta, w_qkv, b_qkv, w_o, b_o, y, B, S, Hq, Hkv, D, eps, causal,
                                workspace, workspace_bytes, stream)


def attn_block_workspace_bytes(B, S, Hq, Hkv, D) -> int:
    return int(lib().attn_block_workspace_bytes(B, S, Hq, Hkv, D))


def attn_splitkv_num_splits(B, Hq, Hkv, Sq, Sk, num_splits=0) -> int:
    return lib().attn_splitkv_num_splits(B, Hq, Hkv, Sq, Sk, num_splits)


def attn_splitkv_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, num_splits=0) -> int:
    return int(lib().attn_splitkv_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, num_splits))


def attn_fwd_window(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, window, sinks, stream) -> int:
    return lib().attn_fwd_window(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, window, sinks, stream)


def attn_fwd_window_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, window, sinks, stream) -> int:
    return lib().attn_fwd_window_f16(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, scale, window, sinks, stream)


def attn_kv_append(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, new_lens, B, S,
                   Hkv, D, page, max_pages, n_pages, cache_kind, rope_table, max_pos, stream) -> int:
    return lib().attn_kv_append(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens,
                                new_lens, B, S, Hkv, D, page, max_pages, n_pages, cache_kind, rope_table, max_pos,
                                stream)


def attn_kv_append_f16(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, new_lens, B,
                       S, Hkv, D, page, max_pages, n_pages, cache_kind, rope_table, max_pos, stream) -> int:
    return lib().attn_kv_append_f16(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens,
                                    new_lens, B, S, Hkv, D, page, max_pages, n_pages, cache_kind, rope_table, max_pos,
                                    stream)


def attn_fwd_paged(q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, o, lse, B, Hq, Hkv,
                   Sq, D, page, max_pages, n_pages, cache_kind, scale, window, sinks, rope_table, max_pos, workspace,
                   workspace_bytes, stream) -> int:
    return lib().attn_fwd_paged(q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, o, lse,
                                B, Hq, Hkv, Sq, D, page, max_pages, n_pages, cache_kind, scale, window, sinks,
                                rope_table, max_pos, workspace, workspace_bytes, stream)


def attn_fwd_paged_f16(q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, o, lse, B, Hq,
                       Hkv, Sq, D, page, max_pages, n_pages, cache_kind, scale, window, sinks, rope_table, max_pos,
                       workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd_paged_f16(q, q_stride, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, o,
                                    lse, B, Hq, Hkv, Sq, D, page, max_pages, n_pages, cache_kind, scale, window, sinks,
                                    rope_table, max_pos, workspace, workspace_bytes, stream)


def attn_paged_workspace_bytes(B, Hq, Hkv, Sq, D, max_keys=0) -> int:
    return int(lib().attn_paged_workspace_bytes(B, Hq, Hkv, Sq, D, max_keys))


def attn_bwd(d_o, q, k, v, o, lse, dq, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, B, Hq, Hkv,
             Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes, stream) -> int:
    return lib().attn_bwd(d_o, q, k, v, o, lse, dq, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride,
                          B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes, stream)


def attn_bwd_f16(d_o, q, k, v, o, lse, dq, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, B, Hq,
                 Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes, stream) -> int:
    return lib().attn_bwd_f16(d_o, q, k, v, o, lse, dq, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride,
                              dv_stride, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace,
                              workspace_bytes, stream)


def attn_bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, mask_kind=0) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, mask_kind))


def attn_rope_axes(q, q_out, q_stride, q_out_stride, k, k_out, k_stride, k_out_stride, B, S, Hq, Hkv, D, rope_table,
                   max_pos, positions, sections, n_axes, inverse, stream) -> int:
    return lib().attn_rope_axes(q, q_out, q_stride, q_out_stride, k, k_out, k_stride, k_out_stride, B, S, Hq, Hkv, D,
                                rope_table, max_pos, positions, sections, n_axes, inverse, stream)


def attn_rope_axes_f16(q, q_out, q_stride, q_out_stride, k, k_out, k_stride, k_out_stride, B, S, Hq, Hkv, D,
                       rope_table, max_pos, positions, sections, n_axes, inverse, stream) -> int:
    return lib().attn_rope_axes_f16(q, q_out, q_stride, q_out_stride, k, k_out, k_stride, k_out_stride, B, S, Hq, Hkv,
                                    D, rope_table, max_pos, positions, sections, n_axes, inverse, stream)


def attn_rope_axes_table(table, max_pos, sections, n_axes, base, stream) -> int:
    return lib().attn_rope_axes_table(table, max_pos, sections, n_axes, float(base), stream)


def attn_checkpoint_store(x, x_stride, codes, scale, B, S, H, D, stream) -> int:
    return lib().attn_checkpoint_store(x, x_stride, codes, scale, B, S, H, D, stream)


def attn_checkpoint_store_f16(x, x_stride, codes, scale, B, S, H, D, stream) -> int:
    return lib().attn_checkpoint_store_f16(x, x_stride, codes, scale, B, S, H, D, stream)


def attn_checkpoint_load(codes, scale, x, x_stride, B, S, H, D, stream) -> int:
    return lib().attn_checkpoint_load(codes, scale, x, x_stride, B, S, H, D, stream)


def attn_checkpoint_load_f16(codes, scale, x, x_stride, B, S, H, D, stream) -> int:
    return lib().attn_checkpoint_load_f16(codes, scale, x, x_stride, B, S, H, D, stream)


def attn_bwd_checkpoint(d_o, q8, k8, v8, q_scale, k_scale, v_scale, dq, dk, dv, dq_stride, dk_stride, dv_stride, B,
                        Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes, stream) -> int:
    return lib().attn_bwd_checkpoint(d_o, q8, k8, v8, q_scale, k_scale, v_scale, dq, dk, dv, dq_stride, dk_stride,
                                     dv_stride, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks,
                                     workspace, workspace_bytes, stream)


def attn_bwd_checkpoint_f16(d_o, q8, k8, v8, q_scale, k_scale, v_scale, dq, dk, dv, dq_stride, dk_stride, dv_stride,
                            B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks, workspace, workspace_bytes,
                            stream) -> int:
    return lib().attn_bwd_checkpoint_f16(d_o, q8, k8, v8, q_scale, k_scale, v_scale, dq, dk, dv, dq_stride, dk_stride,
                                         dv_stride, B, Hq, Hkv, Sq, Sk, D, scale, mask_kind, mask, window, sinks,
                                         workspace, workspace_bytes, stream)


def attn_bwd_checkpoint_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, mask_kind=0) -> int:
    return int(lib().attn_bwd_checkpoint_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, mask_kind))


def attn_last_status(stream) -> int:
    return lib().attn_last_status(stream)


def attn_status_string(code: int) -> str:
    return lib().attn_status_string(int(code)).decode()


def attn_set_wait_timeout_ns(ns: int) -> int:
    return lib().attn_set_wait_timeout_ns(int(ns))


def attn_debug_inject_stall(on: bool) -> int:
    return lib().attn_debug_inject_stall(1 if on else 0)


def attn_abi_version() -> int:
    return lib().attn_abi_version()


# ------------------------------------------------------ torch convenience

def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def attention(q, k, v, *, causal: bool = False, mask=None, scale=None, out=None, lse=None, stream=None):
    """O, LSE = attention(Q, K, V) on (B, S, H, D) bf16 or fp16 CUDA tensors.

    mask: optional FP32 (B, Sq, Sk) additive mask (broadcast over heads).
    scale: None selects 1/sqrt(D). out/lse: optional preallocated outputs.
    bf16 inputs go to attn_fwd, fp16 inputs to attn_fwd_f16.
    """
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q, k, v must be bf16 or fp16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not (t.is_cuda and t.dtype == q.dtype and t.dim() == 4 and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor (B, S, H, D) of q's dtype")
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or v.shape != k.shape:
        raise ValueError("q, k, v shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    kind = (MASK_CAUSAL if causal else MASK_NONE) + (MASK_ADDITIVE if mask is not None else 0)
    mptr = None
    if mask is not None:
        if not (mask.is_cuda and mask.dtype == torch.float32 and mask.is_contiguous()
                and tuple(mask.shape) == (B, Sq, Sk)):
            raise ValueError("mask must be a contiguous FP32 CUDA tensor of shape (B, Sq, Sk)")
        mptr = mask.data_ptr()
    sc = float("nan") if scale is None else float(scale)
    fn = attn_fwd if q.dtype == torch.bfloat16 else attn_fwd_f16
    rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
            B, Hq, Hkv, Sq, Sk, D, sc, kind, mptr, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc)
    return out, lse


def attention_splitkv(q, k, v, *, causal: bool = False, mask=None, scale=None, num_splits: int = 0,
                      workspace=None, out=None, lse=None, stream=None):
    """attention() with the keys split into ranges that are merged afterwards.

    workspace: optional uint8 CUDA tensor of at least attn_splitkv_workspace_bytes
    bytes (allocated here with PyTorch when omitted).
    """
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q, k, v must be bf16 or fp16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not (t.is_cuda and t.dtype == q.dtype and t.dim() == 4 and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor (B, S, H, D) of q's dtype")
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or v.shape != k.shape:
        raise ValueError("q, k, v shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    need = attn_splitkv_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    kind = (MASK_CAUSAL if causal else MASK_NONE) + (MASK_ADDITIVE if mask is not None else 0)
    mptr = None
    if mask is not None:
        if not (mask.is_cuda and mask.dtype == torch.float32 and mask.is_contiguous()
                and tuple(mask.shape) == (B, Sq, Sk)):
            raise ValueError("mask must be a contiguous FP32 CUDA tensor of shape (B, Sq, Sk)")
        mptr = mask.data_ptr()
    sc = float("nan") if scale is None else float(scale)
    fn = attn_fwd_splitkv if q.dtype == torch.bfloat16 else attn_fwd_splitkv_f16
    rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, Sk, D,
            sc, kind, mptr, int(num_splits), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_splitkv")
    return out, lse


def rope_table(max_pos: int, D: int, base: float = 10000.0, *, device=None, stream=None):
    """FP32 (max_pos, D/2, 2) table of {cos, sin}(pos * base^(-2i/D)), built on the GPU."""
    import torch
    table = torch.empty((max_pos, D // 2, 2), dtype=torch.float32, device=device or "cuda")
    rc = attn_rope_table(table.data_ptr(), max_pos, D, base, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_table")
    return table


def rope_apply(x, table, *, pos0: int = 0, out=None, stream=None):
    """Rotate every head vector of a (B, S, H, D) bf16/fp16 CUDA tensor (row s at
    position pos0 + s) into `out` (new tensor by default; may be x itself)."""
    import torch
    if x.dtype not in (torch.bfloat16, torch.float16) or not (x.is_cuda and x.dim() == 4 and x.is_contiguous()):
        raise ValueError("x must be a contiguous 4-D bf16/fp16 CUDA tensor (B, S, H, D)")
    if out is None:
        out = torch.empty_like(x)
    B, S, H, D = x.shape
    fn = attn_rope_apply if x.dtype == torch.bfloat16 else attn_rope_apply_f16
    rc = fn(x.data_ptr(), out.data_ptr(), B, S, H, D, table.data_ptr(), table.shape[0], int(pos0),
            _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_apply")
    return out


def attention_rope(q, k, v, table, *, q_pos0: int = 0, k_pos0: int = 0, k_rot="new", causal: bool = False,
                   mask=None, scale=None, num_splits: int = 1, workspace=None, out=None, lse=None, stream=None):
    """attention(rot(Q), rot(K), V) with the rotary table of rope_table().

    Q is rotated inside the attention kernel at tile load. k_rot: "new" (a
    tensor allocated here receives the rotated keys), a tensor of k's shape
    (may be k itself: rotated in place), or None (k already holds rotated
    keys). num_splits / workspace as for attention_splitkv (1: no split).
    Returns (out, lse) or, when the keys were rotated here, (out, lse, k_rot).
    """
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q, k, v must be bf16 or fp16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not (t.is_cuda and t.dtype == q.dtype and t.dim() == 4 and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor (B, S, H, D) of q's dtype")
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or v.shape != k.shape:
        raise ValueError("q, k, v shapes disagree")
    if not (table.is_cuda and table.dtype == torch.float32 and table.dim() == 3 and table.shape[1:] == (D // 2, 2)
            and table.is_contiguous()):
        raise ValueError("table must be the (max_pos, D/2, 2) FP32 CUDA tensor of rope_table() for this D")
    if isinstance(k_rot, str):
        if k_rot != "new":
            raise ValueError("k_rot must be 'new', a tensor of k's shape, or None")
        k_rot = torch.empty_like(k)
    if k_rot is not None and not (k_rot.is_cuda and k_rot.dtype == k.dtype and k_rot.shape == k.shape
                                  and k_rot.is_contiguous()):
        raise ValueError("k_rot must be a contiguous CUDA tensor of k's shape and dtype")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    need = attn_splitkv_workspace_bytes(B, Hq, Hq, Sq, Sk, D, num_splits)    # rotary tiles never pack heads
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    kind = (MASK_CAUSAL if causal else MASK_NONE) + (MASK_ADDITIVE if mask is not None else 0)
    mptr = None
    if mask is not None:
        if not (mask.is_cuda and mask.dtype == torch.float32 and mask.is_contiguous()
                and tuple(mask.shape) == (B, Sq, Sk)):
            raise ValueError("mask must be a contiguous FP32 CUDA tensor of shape (B, Sq, Sk)")
        mptr = mask.data_ptr()
    sc = float("nan") if scale is None else float(scale)
    fn = attn_fwd_rope if q.dtype == torch.bfloat16 else attn_fwd_rope_f16
    rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, Sk, D,
            sc, kind, mptr, table.data_ptr(), table.shape[0], int(q_pos0), int(k_pos0),
            None if k_rot is None else k_rot.data_ptr(), int(num_splits),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_rope")
    return (out, lse) if k_rot is None else (out, lse, k_rot)


def attention_host(q, k, v, *, causal: bool = False, mask=None, scale=None, out=None, lse=None, workspace=None,
                   device=None, stream=None):
    """attention() for (B, S, H, D) bf16/fp16 tensors in host memory (pin them
    for full speed): copies in, computes and copies back in a pipeline on the
    GPU. Returns (out, lse) in host memory, written once `stream` (default: the
    current stream of `device`) has been synchronised; this function does not
    synchronise. workspace: optional uint8 CUDA tensor of at least
    attn_fwd_host_workspace_bytes bytes (allocated here when omitted).
    """
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("q, k, v must be bf16 or fp16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not (t.device.type == "cpu" and t.dtype == q.dtype and t.dim() == 4 and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous 4-D host tensor (B, S, H, D) of q's dtype")
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if (Bk, Dk) != (B, D) or v.shape != k.shape:
        raise ValueError("q, k, v shapes disagree")
    pin = q.is_pinned()
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=pin)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, pin_memory=pin)
    kind = (MASK_CAUSAL if causal else MASK_NONE) + (MASK_ADDITIVE if mask is not None else 0)
    mptr = None
    if mask is not None:
        if not (mask.device.type == "cpu" and mask.dtype == torch.float32 and mask.is_contiguous()
                and tuple(mask.shape) == (B, Sq, Sk)):
            raise ValueError("mask must be a contiguous FP32 host tensor of shape (B, Sq, Sk)")
        mptr = mask.data_ptr()
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    need = attn_fwd_host_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, kind)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    sc = float("nan") if scale is None else float(scale)
    fn = attn_fwd_host if q.dtype == torch.bfloat16 else attn_fwd_host_f16
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, Sk, D, sc,
                kind, mptr, workspace.data_ptr(), workspace.numel() * workspace.element_size(), s.cuda_stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_host")
    return out, lse


def _bf16_cuda(name, t, dim=None):
    import torch
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous() and (dim is None or t.dim() == dim)):
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor" + (f" with {dim} dimensions" if dim else ""))


def linear(a, w, bias=None, residual=None, *, out=None, stream=None):
    """out = a w^T (+ bias) (+ residual) for bf16 CUDA tensors a (M, K), w (N, K)."""
    import torch
    _bf16_cuda("a", a, 2)
    _bf16_cuda("w", w, 2)
    M, K = a.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("a and w disagree on K")
    for name, t, shape in (("bias", bias, (N,)), ("residual", residual, (M, N))):
        if t is not None:
            _bf16_cuda(name, t)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    rc = attn_linear(a.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
                     None if residual is None else residual.data_ptr(), out.data_ptr(), M, N, K, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_linear")
    return out


def layernorm(x, gamma, beta, eps: float = 1e-5, *, out=None, stream=None):
    """Row-wise LayerNorm over the last dimension of a bf16 CUDA tensor."""
    import torch
    for name, t in (("x", x), ("gamma", gamma), ("beta", beta)):
        _bf16_cuda(name, t)
    H = x.shape[-1]
    M = x.numel() // H if H else 0
    if out is None:
        out = torch.empty_like(x)
    rc = attn_layernorm(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), out.data_ptr(), M, H, float(eps),
                        _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_layernorm")
    return out


def attention_qkvpacked(qkv, Hq: int, Hkv: int, D: int, *, causal: bool = False, scale=None, out=None, lse=None,
                        stream=None):
    """Self-attention on a packed (B, S, (Hq + 2 Hkv) D) bf16 tensor [q | k | v]."""
    import torch
    _bf16_cuda("qkv", qkv, 3)
    B, S, F = qkv.shape
    if F != (Hq + 2 * Hkv) * D:
        raise ValueError("qkv's last dimension must be (Hq + 2 Hkv) D")
    if out is None:
        out = torch.empty((B, S, Hq, D), dtype=torch.bfloat16, device=qkv.device)
    if lse is None:
        lse = torch.empty((B, Hq, S), dtype=torch.float32, device=qkv.device)
    sc = float("nan") if scale is None else float(scale)
    rc = attn_fwd_qkvpacked(qkv.data_ptr(), out.data_ptr(), lse.data_ptr(), B, S, Hq, Hkv, D, sc,
                            MASK_CAUSAL if causal else MASK_NONE, None, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_qkvpacked")
    return out, lse


def attention_block(x, ln_gamma, ln_beta, w_qkv, b_qkv, w_o, b_o, *, Hq: int, Hkv: int, D: int,
                    causal: bool = True, eps: float = 1e-5, out=None, workspace=None, stream=None):
    """The attention block (LayerNorm, QKV projection, attention, output
    projection, residual) on x (B, S, Hq*D) bf16 CUDA; returns y."""
    import torch
    for name, t in (("x", x), ("ln_gamma", ln_gamma), ("ln_beta", ln_beta), ("w_qkv", w_qkv), ("b_qkv", b_qkv),
                    ("w_o", w_o), ("b_o", b_o)):
        _bf16_cuda(name, t)
    B, S, H = x.shape
    F = (Hq + 2 * Hkv) * D
    if H != Hq * D or tuple(w_qkv.shape) != (F, H) or tuple(b_qkv.shape) != (F,) or tuple(w_o.shape) != (H, H) \
            or tuple(b_o.shape) != (H,) or tuple(ln_gamma.shape) != (H,) or tuple(ln_beta.shape) != (H,):
        raise ValueError("attention block shapes disagree")
    if out is None:
        out = torch.empty_like(x)
    need = attn_block_workspace_bytes(B, S, Hq, Hkv, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    rc = attn_block_fwd(x.data_ptr(), ln_gamma.data_ptr(), ln_beta.data_ptr(), w_qkv.data_ptr(), b_qkv.data_ptr(),
                        w_o.data_ptr(), b_o.data_ptr(), out.data_ptr(), B, S, Hq, Hkv, D, float(eps),
                        1 if causal else 0, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_block_fwd")
    return out


# ------------------------------------------- windows and the paged key/value cache
# These wrappers run once per layer and decode step, so the usual call (tensors as
# they should be, on the current device and stream) goes through the native module
# _binding, from one interpreter step to the C ABI. What it leaves alone comes to
# the checks here: one condition over everything, and the message sought only once
# it has failed.

_torch = None
_native = None
_NAN = float("nan")


def _bind():
    """torch and the native module, imported at first use (the C ABI above needs neither)."""
    global _torch, _native
    import torch
    lib()
    if not os.path.exists(_build.BINDING):
        raise RuntimeError(
            f"{_build.BINDING} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    from . import _binding
    _native = _binding
    _torch = torch
    return torch


def _token_stride(name, t, at):
    """Elements from token to token of a (B, S, H, D) tensor on device `at` whose tokens are evenly spaced and
    contiguous inside (a contiguous tensor, or a slice of a packed projection)."""
    if at < 0 or t.get_device() != at:
        raise ValueError(f"{name} must be a CUDA tensor on the other tensors' device")
    B, S, H, D = t.shape
    if t.is_contiguous():
        return H * D
    sb, ss, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if S == 1:
        return sb if B > 1 else max(ss, H * D)
    if B > 1 and sb != S * ss:
        raise ValueError(f"{name}: the tokens of the flattened (B, S) must be evenly spaced")
    return ss


def _device_of(x, xname):
    """Index of a CUDA tensor's device; checks its type and rank too."""
    torch = _torch or _bind()
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float16:
        raise ValueError(f"{xname} must be bf16 or fp16")
    if x.dim() != 4:
        raise ValueError(f"{xname} must have 4 dimensions (B, S, H, D)")
    return x.get_device()


def _enter_device(at):
    """Makes device `at` current (the C ABI works on the current device); returns the one to go back to, or None."""
    now = _torch.cuda.current_device()
    if now == at:
        return None
    _torch.cuda.set_device(at)
    return now


def _stream_on(at, stream):
    """Handle of `stream`, or of device `at`'s current stream."""
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)     # current_stream() without making a Stream object
    return _torch.cuda.current_stream(at).cuda_stream if raw is None else raw(at)


_INT_MAX = 2 ** 31 - 1


def _count(name, n):
    """A window or a number of sinks as a C int: past its range it means all keys."""
    if n < 0:
        raise ValueError(f"{name} must not be negative")
    return n if n <= _INT_MAX else _INT_MAX


def _new(shape, dtype, like, stream):
    t = _torch.empty(shape, dtype=dtype, device=like.device)
    if stream is not None:
        t.record_stream(stream)                    # allocated on the current stream, used on another
    return t


@functools.lru_cache(maxsize=1024)
def _paged_workspace_size(at, B, Hq, Hkv, Sq, D, max_keys):
    return _lib.attn_paged_workspace_bytes(B, Hq, Hkv, Sq, D, max_keys) or 1      # (device `at` is current)


_HELD_BYTES = 32 << 20                              # larger workspaces (long chunks of queries) are a call's own


class _Held(threading.local):
    """Workspace of a thread's calls on a device's default stream, as {device: tensor}. Calls of one thread on
    one stream run in order, so they may share it; another thread could enqueue between a call's two kernels, another
    stream run beside them, and a captured call is replayed at any time, so all those get their own."""

    def __init__(self):
        self.by_device = {}


_held = _Held()


def _workspace(q, at, size, handle, stream):
    """(address, bytes, the tensor to keep until the call is enqueued)."""
    if stream is not None or handle or size > _HELD_BYTES or _torch.cuda.is_current_stream_capturing():
        t = _new(size, _torch.uint8, q, stream)
        return t.data_ptr(), size, t
    held = _held.by_device.get(at)
    if held is None or held.numel() < size:
        held = _held.by_device[at] = _torch.empty(size, dtype=_torch.uint8, device=q.device)
    return held.data_ptr(), held.numel(), held


def _outputs(q, at, out, lse, stream):
    """The given outputs of an attention over q (B, Sq, Hq, D), checked, or new ones."""
    shape = q.shape
    B, Sq, Hq, _ = shape
    if out is None:
        out = _new(shape, q.dtype, q, stream)
    elif out.dtype is not q.dtype or out.get_device() != at or out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous (B, Sq, Hq, D) tensor of q's type and device")
    if lse is None:
        lse = _new((B, Hq, Sq), _torch.float32, q, stream)
    elif (lse.dtype is not _torch.float32 or lse.get_device() != at or lse.shape != (B, Hq, Sq)
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous FP32 (B, Hq, Sq) tensor on q's device")
    return out, lse


def attention_window(q, k, v, *, window: int, sinks: int = 0, scale=None, out=None, lse=None, stream=None):
    """O, LSE = causal attention with a sliding window on (B, S, H, D) bf16 or fp16 CUDA tensors.

    The query at position p (its row plus Sk - Sq) sees the last `window` keys up to p, its own included, and the first
    `sinks` keys. scale: None selects 1/sqrt(D). out/lse: optional preallocated outputs.
    """
    if _native is not None and stream is None:
        done = _native.attention_window(q, k, v, window, sinks, scale, out, lse)
        if done is not None:
            if done.__class__ is int:
                raise AttnError(done, "attn_fwd_window")
            return done
    at = _device_of(q, "q")
    qs, ks = q.shape, k.shape
    B, Sq, Hq, D = qs
    for name, t in (("q", q), ("k", k), ("v", v)):
        if at < 0 or t.get_device() != at or t.dtype is not q.dtype or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor (B, S, H, D) of q's dtype and device")
    if ks[0] != B or ks[3] != D or v.shape != ks:
        raise ValueError("q, k, v shapes disagree")
    L = lib()
    back = _enter_device(at)
    try:
        out, lse = _outputs(q, at, out, lse, stream)
        fn = L.attn_fwd_window if q.dtype is _torch.bfloat16 else L.attn_fwd_window_f16
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, ks[2], Sq, ks[1], D,
                _NAN if scale is None else scale, _count("window", window), _count("sinks", sinks),
                _stream_on(at, stream))
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_window")
    return out, lse


def _cache_args(x, xname, at, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, lens, lens_name, table):
    """Checks what the cache's calls share; returns their common arguments."""
    torch = _torch
    shape, dtype = k_cache.shape, k_cache.dtype
    i32, f32 = torch.int32, torch.float32
    B = x.shape[0]
    ks = vs = nl = rope = None
    max_pos = 0
    if len(shape) == 4 and block_table.dim() == 2:
        n_pages, Hkv, page, D = shape
        max_pages = block_table.shape[1]
        kind = CACHE_16BIT
        ok = (v_cache.shape == shape and v_cache.dtype is dtype and k_cache.get_device() == at
              and v_cache.get_device() == at and k_cache.is_contiguous() and v_cache.is_contiguous()
              and block_table.dtype is i32 and block_table.shape[0] == B and block_table.get_device() == at
              and block_table.is_contiguous()
              and kv_lens.dtype is i32 and kv_lens.shape == (B,) and kv_lens.get_device() == at
              and kv_lens.is_contiguous())
        if dtype is torch.float8_e4m3fn:
            kind, pair = CACHE_E4M3, (n_pages, Hkv)
            ok = (ok and k_scale is not None and v_scale is not None
                  and k_scale.dtype is f32 and k_scale.shape == pair and k_scale.get_device() == at
                  and k_scale.is_contiguous()
                  and v_scale.dtype is f32 and v_scale.shape == pair and v_scale.get_device() == at
                  and v_scale.is_contiguous())
            if ok:
                ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
        else:
            ok = ok and dtype is x.dtype and k_scale is None and v_scale is None
        if lens is not None:
            ok = (ok and lens.dtype is i32 and lens.shape == (B,) and lens.get_device() == at and lens.is_contiguous())
            nl = lens.data_ptr()
        if table is not None:
            ok = (ok and table.dtype is f32 and table.dim() == 3 and table.shape[1] == D // 2 and table.shape[2] == 2
                  and table.shape[0] > 0 and table.get_device() == at and table.is_contiguous())
            rope, max_pos = table.data_ptr(), table.shape[0]
        if ok:
            return (kind, ks, vs, block_table.data_ptr(), kv_lens.data_ptr(), nl, Hkv, D, page, max_pages, n_pages, rope,
                    max_pos)
    raise ValueError(_cache_fault(x, xname, at, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, lens, lens_name,
                                  table))


def _cache_fault(x, xname, at, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, lens, lens_name, table):
    """What is wrong with the arguments that _cache_args refuses."""
    torch = _torch
    if (k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.dtype is not k_cache.dtype
            or k_cache.get_device() != at or v_cache.get_device() != at or not k_cache.is_contiguous()
            or not v_cache.is_contiguous()):
        return f"k_cache and v_cache must be contiguous (n_pages, Hkv, page, D) tensors of one type on {xname}'s device"
    B = x.shape[0]
    for name, t, want in (("block_table", block_table, (B, block_table.shape[-1]) if block_table.dim() else (B, 1)),
                          ("kv_lens", kv_lens, (B,)), (lens_name, lens, (B,))):
        if t is not None and (t.dtype is not torch.int32 or tuple(t.shape) != want or t.get_device() != at
                              or not t.is_contiguous()):
            return f"{name} must be a contiguous int32 CUDA tensor of shape {want} on the other tensors' device"
    if k_cache.dtype is not torch.float8_e4m3fn and k_cache.dtype is not x.dtype:
        return f"the cache must be float8_e4m3fn or of {xname}'s type"
    if k_cache.dtype is x.dtype and (k_scale is not None or v_scale is not None):
        return "a 16-bit cache has no scales"
    if table is not None and (table.dtype is not torch.float32 or table.dim() != 3
                              or tuple(table.shape[1:]) != (k_cache.shape[3] // 2, 2) or table.shape[0] == 0
                              or table.get_device() != at
                              or not table.is_contiguous()):
        return "table must be the (max_pos, D/2, 2) FP32 CUDA tensor of rope_table() for this D"
    return ("k_scale and v_scale must be contiguous FP32 CUDA tensors of shape (n_pages, Hkv): an 8-bit cache needs its "
            "scales")


def kv_append(k, v, k_cache, v_cache, block_table, kv_lens, *, new_lens=None, k_scale=None, v_scale=None, table=None,
              stream=None):
    """Write a step's keys and values (B, S, Hkv, D) into a paged cache, in place.

    k, v: bf16/fp16 CUDA tensors, contiguous or evenly spaced slices of a packed projection.
    k_cache, v_cache: (n_pages, Hkv, page, D), of k's type or float8_e4m3fn; the latter with k_scale, v_scale
    (n_pages, Hkv) FP32, which the call updates. block_table (B, max_pages), kv_lens (B) and new_lens (B, default S
    each) are int32; kv_lens counts the step's tokens already: token s of sequence b goes to position
    kv_lens[b] - new_lens[b] + s. table: rope_table() to rotate the keys to their positions, or None.
    """
    if _native is not None and stream is None:
        rc = _native.kv_append(k, v, k_cache, v_cache, block_table, kv_lens, new_lens, k_scale, v_scale, table)
        if rc is not None:
            if rc:
                raise AttnError(rc, "attn_kv_append")
            return
    at = _device_of(k, "k")
    kind, ks, vs, bt, kl, nl, Hkv, D, page, max_pages, n_pages, rope, max_pos = _cache_args(
        k, "k", at, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, new_lens, "new_lens", table)
    shape, dtype = k.shape, k.dtype
    B, S, H, Dk = shape
    if v.dtype is not dtype or v.shape != shape or H != Hkv or Dk != D:
        raise ValueError("k and v must be (B, S, Hkv, D) tensors of one type, with the cache's Hkv and D")
    k_stride, v_stride = _token_stride("k", k, at), _token_stride("v", v, at)
    L = _lib or lib()
    fn = L.attn_kv_append if dtype is _torch.bfloat16 else L.attn_kv_append_f16
    back = _enter_device(at)
    try:
        rc = fn(k.data_ptr(), v.data_ptr(), k_stride, v_stride, k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, bt, kl,
                nl, B, S, Hkv, D, page, max_pages, n_pages, kind, rope, max_pos, _stream_on(at, stream))
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_kv_append")


def attention_paged(q, k_cache, v_cache, block_table, kv_lens, *, q_lens=None, k_scale=None, v_scale=None, table=None,
                    window: int = 0, sinks: int = 0, scale=None, out=None, lse=None, workspace=None, stream=None):
    """O, LSE = causal attention of a step's queries (B, Sq, Hq, D) over a paged cache (see kv_append).

    Query i of sequence b sits at position kv_lens[b] - q_lens[b] + i (q_lens: default Sq each) and sees the keys up
    to it; window > 0: only the last `window` of them and the first `sinks` tokens. table: rope_table() to rotate the
    queries to their positions, or None. Rows i >= q_lens[b] of out and lse are not written. workspace: optional
    uint8 CUDA tensor of at least attn_paged_workspace_bytes bytes; when omitted, one that the calling thread keeps for
    the device's default stream, or, on another stream or under capture, a new one.
    """
    if _native is not None and stream is None:
        done = _native.attention_paged(q, k_cache, v_cache, block_table, kv_lens, q_lens, k_scale, v_scale, table, window,
                                       sinks, scale, out, lse, workspace, _held.by_device.get(q.get_device()), _HELD_BYTES)
        if done is not None:
            if done.__class__ is int:
                raise AttnError(done, "attn_fwd_paged")
            return done
    at = _device_of(q, "q")
    kind, ks, vs, bt, kl, nl, Hkv, D, page, max_pages, n_pages, rope, max_pos = _cache_args(
        q, "q", at, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_lens, "q_lens", table)
    q_stride = _token_stride("q", q, at)
    B, Sq, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q and the cache disagree on D")
    L = _lib or lib()
    back = _enter_device(at)
    try:
        out, lse = _outputs(q, at, out, lse, stream)
        handle = _stream_on(at, stream)
        if workspace is None:
            ws, size, keep = _workspace(q, at, _paged_workspace_size(at, B, Hq, Hkv, Sq, D, max_pages * page), handle,
                                        stream)
        else:
            if workspace.get_device() != at or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
            ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        fn = L.attn_fwd_paged if q.dtype is _torch.bfloat16 else L.attn_fwd_paged_f16
        rc = fn(q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, bt, kl, nl, out.data_ptr(),
                lse.data_ptr(), B, Hq, Hkv, Sq, D, page, max_pages, n_pages, kind, _NAN if scale is None else scale,
                _count("window", window), _count("sinks", sinks), rope, max_pos, ws, size, handle)
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_fwd_paged")
    return out, lse


# ------------------------------------------------------------ the backward pass

def _mask_arg(mask, at, shape):
    """Address of an additive mask, checked, or None."""
    if mask is None:
        return None
    if mask.dtype is not _torch.float32 or mask.get_device() != at or mask.shape != shape or not mask.is_contiguous():
        raise ValueError("mask must be a contiguous FP32 CUDA tensor of shape (B, Sq, Sk) on q's device")
    return mask.data_ptr()


def _gradient(name, t, like, at, stream):
    """(tensor, token stride): the given gradient, checked, or a new contiguous one of `like`'s shape and type."""
    if t is None:
        t = _new(like.shape, like.dtype, like, stream)
    elif t.dtype is not like.dtype or t.get_device() != at or t.shape != like.shape:
        raise ValueError(f"{name} must have the shape, type and device of the tensor it belongs to")
    return t, _token_stride(name, t, at)


def _own_workspace(workspace, size, like, at, stream):
    """The given workspace, checked, or a new one of `size` bytes."""
    if workspace is None:
        return _new((max(size, 1),), _torch.uint8, like, stream)
    if workspace.get_device() != at or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
    return workspace


def _attention_mask(causal, mask, window):
    """The mask kind of a backward pass; a window needs a causal one."""
    if window and (not causal or mask is not None):
        raise ValueError("a window needs causal=True and no additive mask")
    return (MASK_CAUSAL if causal else MASK_NONE) + (MASK_ADDITIVE if mask is not None else 0)


def attention_backward(d_o, q, k, v, o, lse, *, causal: bool = False, mask=None, window: int = 0, sinks: int = 0,
                       scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV = the gradients of attention(), attention_qkvpacked() or, with window > 0, attention_window().

    d_o: the gradient of the output, and o (B, Sq, Hq, D) and lse (B, Hq, Sq) as the forward call returned them. q
    (B, Sq, Hq, D), k, v (B, Sk, Hkv, D): bf16 or fp16 CUDA tensors, contiguous or evenly spaced slices of a packed
    projection; so may be dq, dk, dv (new contiguous tensors by default), which overlap no input. causal, mask, window,
    sinks, scale: those of the forward call; the mask has no gradient. workspace: optional uint8 CUDA tensor of at least
    attn_bwd_workspace_bytes bytes.
    """
    if _native is not None and stream is None:
        done = _native.attention_backward(d_o, q, k, v, o, lse, causal, mask, window, sinks, scale, dq, dk, dv, workspace)
        if done is not None:
            if done.__class__ is int:
                raise AttnError(done, "attn_bwd")
            return done
    at = _device_of(q, "q")
    for name, t in (("k", k), ("v", v), ("o", o), ("d_o", d_o)):
        if t.dtype is not q.dtype or t.dim() != 4:
            raise ValueError(f"{name} must be a 4-D tensor (B, S, H, D) of q's type")
    q_stride, k_stride, v_stride = _token_stride("q", q, at), _token_stride("k", k, at), _token_stride("v", v, at)
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != D or v.shape != k.shape:
        raise ValueError("q, k, v shapes disagree")
    for name, t in (("o", o), ("d_o", d_o)):
        if t.shape != q.shape or t.get_device() != at or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of q's shape and device")
    if (lse.dtype is not _torch.float32 or lse.get_device() != at or lse.shape != (B, Hq, Sq)
            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous FP32 (B, Hq, Sq) tensor on q's device")
    window, sinks = _count("window", window), _count("sinks", sinks)
    kind = _attention_mask(causal, mask, window)
    L = _lib or lib()
    back = _enter_device(at)
    try:
        dq, dq_stride = _gradient("dq", dq, q, at, stream)
        dk, dk_stride = _gradient("dk", dk, k, at, stream)
        dv, dv_stride = _gradient("dv", dv, v, at, stream)
        ws = _own_workspace(workspace, L.attn_bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, kind), q, at, stream)
        fn = L.attn_bwd if q.dtype is _torch.bfloat16 else L.attn_bwd_f16
        rc = fn(d_o.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dq.data_ptr(),
                dk.data_ptr(), dv.data_ptr(), q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, B, Hq, Hkv, Sq,
                Sk, D, _NAN if scale is None else scale, kind, _mask_arg(mask, at, (B, Sq, Sk)), window, sinks,
                ws.data_ptr(), ws.numel() * ws.element_size(), _stream_on(at, stream))
    finally:
        if back is not None:
            _torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_bwd")
    return dq, dk, dv


# --------------------------------------- rotary positions with several axes

def _sections(sections):
    """The pairs of each axis as a C array (kept alive by the caller), and their number."""
    sections = tuple(sections)
    if not 1 <= len(sections) <= 4 or any(not 0 <= n <= 512 for n in sections):
        raise ValueError("sections must be 1 to 4 numbers of pairs, each 0 to 512")
    return (ctypes.c_int * len(sections))(*sections), len(sections)


def rope_axes_table(max_pos: int, sections, base: float = 10000.0, *, device=None, stream=None):
    """FP32 (max_pos, sum(sections), 2) table of {cos, sin}(pos * base^(-j/n)) for pair j of an axis of n pairs.

    Each axis has the frequencies of a head of its own size; rope_table() is the table of the other kind, in which a
    pair's frequency goes by its number in the head vector.
    """
    torch = _torch or _bind()
    axes, n = _sections(sections)
    device = torch.device(device or "cuda")
    at = torch.cuda.current_device() if device.index is None else device.index
    back = _enter_device(at)
    try:
        table = _new((max_pos, sum(axes), 2), torch.float32, torch.empty(0, device=device), stream)
        rc = attn_rope_axes_table(table.data_ptr(), max_pos, axes, n, base, _stream_on(at, stream))
    finally:
        if back is not None:
            torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_rope_axes_table")
    return table


def rope_axes(q, k, table, positions, sections, *, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Turn queries (B, S, Hq, D) and keys (B, S, Hkv, D) to positions of several axes; k may be None.

    sections: pairs of a head vector that each axis turns, in order (D/2 together); positions: int32 CUDA tensor
    (B, S, len(sections)); table: rope_table() or rope_axes_table() for this D. inverse: by the opposite angle, the way
    of a gradient. q, k: bf16 or fp16, contiguous or evenly spaced slices of a packed projection; so may be q_out and
    k_out (new contiguous tensors by default; q and k themselves: in place). Returns (q_out, k_out), or q_out without k.
    """
    if _native is not None and stream is None:
        done = _native.rope_axes(q, k, table, positions, sections, inverse, q_out, k_out)
        if done is not None:
            if done.__class__ is int:
                raise AttnError(done, "attn_rope_axes")
            return done
    at = _device_of(q, "q")
    torch = _torch
    B, S, Hq, D = q.shape
    axes, n = _sections(sections)
    if sum(axes) * 2 != D:
        raise ValueError("sections must add up to D/2")
    if (positions.dtype is not torch.int32 or positions.shape != (B, S, n) or positions.get_device() != at
            or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 CUDA tensor of shape (B, S, len(sections)) on q's device")
    if (table.dtype is not torch.float32 or table.dim() != 3 or tuple(table.shape[1:]) != (D // 2, 2)
            or table.shape[0] == 0 or table.get_device() != at or not table.is_contiguous()):
        raise ValueError("table must be the (max_pos, D/2, 2) FP32 CUDA tensor of rope_table() or rope_axes_table() for this D")
    q_stride, Hkv, k_stride, ko_stride, k_in = _token_stride("q", q, at), 0, 0, 0, None
    if k is not None:
        if k.dtype is not q.dtype or k.dim() != 4 or k.shape[0] != B or k.shape[1] != S or k.shape[3] != D:
            raise ValueError("k must be a (B, S, Hkv, D) tensor of q's type, B, S and D")
        Hkv, k_stride, k_in = k.shape[2], _token_stride("k", k, at), k.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    fn = attn_rope_axes if q.dtype is torch.bfloat16 else attn_rope_axes_f16
    back = _enter_device(at)
    try:
        q_out, qo_stride = _gradient("q_out", q_out, q, at, stream)
        if k is not None:
            k_out, ko_stride = _gradient("k_out", k_out, k, at, stream)
        rc = fn(q.data_ptr(), q_out.data_ptr(), q_stride, qo_stride, k_in, None if k is None else k_out.data_ptr(), k_stride,
                ko_stride, B, S, Hq, Hkv, D, table.data_ptr(), table.shape[0], positions.data_ptr(), axes, n,
                1 if inverse else 0, _stream_on(at, stream))
    finally:
        if back is not None:
            torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_rope_axes")
    return q_out if k is None else (q_out, k_out)


# ------------------------------------------------- activation checkpoints in 8 bits

def checkpoint_store(x, *, codes=None, scale=None, stream=None):
    """(codes, scale) of a bf16 or fp16 CUDA tensor x (B, S, H, D), contiguous or an evenly spaced slice.

    codes: float8_e4m3fn (B, S, H, D), value / scale; scale: FP32 (B, S, H), a power of two for each head vector, the
    smallest with max |x| <= 448 * scale.
    """
    if _native is not None and stream is None:
        done = _native.checkpoint_store(x, codes, scale)
        if done is not None:
            if done.__class__ is int:
                raise AttnError(done, "attn_checkpoint_store")
            return done
    at = _device_of(x, "x")
    torch = _torch
    B, S, H, D = x.shape
    x_stride = _token_stride("x", x, at)
    if codes is not None and (codes.dtype is not torch.float8_e4m3fn or codes.shape != x.shape or codes.get_device() != at
                              or not codes.is_contiguous()):
        raise ValueError("codes must be a contiguous float8_e4m3fn tensor of x's shape and device")
    if scale is not None and (scale.dtype is not torch.float32 or scale.shape != (B, S, H) or scale.get_device() != at
                              or not scale.is_contiguous()):
        raise ValueError("scale must be a contiguous FP32 (B, S, H) tensor on x's device")
    fn = attn_checkpoint_store if x.dtype is torch.bfloat16 else attn_checkpoint_store_f16
    back = _enter_device(at)
    try:
        if codes is None:
            codes = _new((B, S, H, D), torch.float8_e4m3fn, x, stream)
        if scale is None:
            scale = _new((B, S, H), torch.float32, x, stream)
        rc = fn(x.data_ptr(), x_stride, codes.data_ptr(), scale.data_ptr(), B, S, H, D, _stream_on(at, stream))
    finally:
        if back is not None:
            torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_checkpoint_store")
    return codes, scale


def _checkpoint(name, pair, at, shape=None):
    """(codes, scale) of a checkpoint, checked; `at` None: any device."""
    torch = _torch
    codes, scale = pair
    if (codes.dtype is not torch.float8_e4m3fn or codes.dim() != 4 or (shape is not None and codes.shape != shape)
            or codes.get_device() < 0 or (at is not None and codes.get_device() != at) or not codes.is_contiguous()):
        raise ValueError(f"{name}: codes must be a contiguous float8_e4m3fn CUDA tensor (B, S, H, D)")
    if (scale.dtype is not torch.float32 or scale.shape != codes.shape[:3] or scale.get_device() != codes.get_device()
            or not scale.is_contiguous()):
        raise ValueError(f"{name}: scale must be a contiguous FP32 (B, S, H) tensor on the codes' device")
    return codes, scale


def checkpoint_load(codes, scale, dtype=None, *, out=None, stream=None):
    """The tensor (B, S, H, D) of a checkpoint in bf16 (the default) or fp16: code * scale."""
    torch = _torch or _bind()
    codes, scale = _checkpoint("checkpoint", (codes, scale), None)
    at = codes.get_device()
    dtype = (torch.bfloat16 if out is None else out.dtype) if dtype is None else dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("dtype must be bf16 or fp16")
    if out is not None and (out.dtype is not dtype or out.shape != codes.shape):
        raise ValueError("out must be a tensor of the codes' shape and of dtype")
    B, S, H, D = codes.shape
    fn = attn_checkpoint_load if dtype is torch.bfloat16 else attn_checkpoint_load_f16
    back = _enter_device(at)
    try:
        if out is None:
            out = _new((B, S, H, D), dtype, codes, stream)
        rc = fn(codes.data_ptr(), scale.data_ptr(), out.data_ptr(), _token_stride("out", out, at), B, S, H, D,
                _stream_on(at, stream))
    finally:
        if back is not None:
            torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_checkpoint_load")
    return out


def attention_backward_checkpoint(d_o, q, k, v, *, causal: bool = False, mask=None, window: int = 0, sinks: int = 0,
                                  scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """attention_backward() from 8-bit checkpoints: q, k, v are the (codes, scale) pairs of checkpoint_store().

    They are widened to d_o's type, o and lse are computed again, and the gradients are those at the widened tensors.
    workspace: optional uint8 CUDA tensor of at least attn_bwd_checkpoint_workspace_bytes bytes; it holds all of that.
    Other arguments as for attention_backward().
    """
    at = _device_of(d_o, "d_o")
    torch = _torch
    if at < 0 or not d_o.is_contiguous():
        raise ValueError("d_o must be a contiguous CUDA tensor (B, Sq, Hq, D)")
    q8, qs = _checkpoint("q", q, at, d_o.shape)
    k8, ks = _checkpoint("k", k, at)
    B, Sq, Hq, D = d_o.shape
    Sk, Hkv = k8.shape[1], k8.shape[2]
    if k8.shape[0] != B or k8.shape[3] != D:
        raise ValueError("q, k, v shapes disagree")
    v8, vs = _checkpoint("v", v, at, k8.shape)
    window, sinks = _count("window", window), _count("sinks", sinks)
    kind = _attention_mask(causal, mask, window)
    L = _lib or lib()
    back = _enter_device(at)
    try:
        dq, dq_stride = _gradient("dq", dq, d_o, at, stream)
        pair = []
        for name, t in (("dk", dk), ("dv", dv)):
            if t is None:
                t = _new(k8.shape, d_o.dtype, d_o, stream)
            elif t.dtype is not d_o.dtype or t.get_device() != at or t.shape != k8.shape:
                raise ValueError(f"{name} must be a (B, Sk, Hkv, D) tensor of d_o's type and device")
            pair.append((t, _token_stride(name, t, at)))
        (dk, dk_stride), (dv, dv_stride) = pair
        ws = _own_workspace(workspace, L.attn_bwd_checkpoint_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, kind), d_o, at, stream)
        fn = L.attn_bwd_checkpoint if d_o.dtype is torch.bfloat16 else L.attn_bwd_checkpoint_f16
        rc = fn(d_o.data_ptr(), q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), qs.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dq_stride, dk_stride, dv_stride, B, Hq, Hkv, Sq, Sk, D,
                _NAN if scale is None else scale, kind, _mask_arg(mask, at, (B, Sq, Sk)), window, sinks, ws.data_ptr(),
                ws.numel() * ws.element_size(), _stream_on(at, stream))
    finally:
        if back is not None:
            torch.cuda.set_device(back)
    if rc:
        raise AttnError(rc, "attn_bwd_checkpoint")
    return dq, dk, dv
