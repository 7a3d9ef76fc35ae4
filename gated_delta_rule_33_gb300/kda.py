"""ctypes binding for libkda (include/kda.h): argument marshalling only.

Each ``kda_*`` function takes torch tensors that already live on the GPU,
passes their device pointers and sizes to the C entry point of the same name
on the current torch stream, and raises ``KDAError`` on a non-OK status.
``gate``/``prefill``/``decode`` are conveniences that allocate the outputs
with torch and call the same entry points.  Nothing here computes any part of
KDA; if libkda.so is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading
from typing import Optional, Tuple

import torch

from . import _build

KDA_BF16 = 0
KDA_FP32 = 1
KDA_FP8_E4M3 = 2
KDA_ALOG_PER_HEAD = 0
KDA_ALOG_PER_CHANNEL = 1
KDA_ALOG_PER_HEAD_CHANNEL = 2

_STATUS_NAMES = {
    0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED_SHAPE",
    3: "KDA_ERR_UNSUPPORTED_DTYPE", 4: "KDA_ERR_MISALIGNED", 5: "KDA_ERR_WORKSPACE_TOO_SMALL",
    6: "KDA_ERR_CUDA", 7: "KDA_ERR_DEVICE_TIMEOUT", 8: "KDA_ERR_NONFINITE",
    9: "KDA_ERR_NOT_IMPLEMENTED", 10: "KDA_ERR_NO_DEVICE", 11: "KDA_ERR_DECAY_RANGE",
}


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {_STATUS_NAMES.get(self.status, self.status)}")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libkda.so for sm_103a (in-tree)."""
    return _build.build(force=force, verbose=verbose)


def load():
    """Load libkda.so (it must have been built); declares every entry point."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libkda.so is not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        lib.kda_version.argtypes = []
        lib.kda_version.restype = I
        lib.kda_status_string.argtypes = [I]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_gate_fused.argtypes = [P, I, P, I, P, I, P, P, P, I64, I, I, P]
        lib.kda_gate_fused.restype = I
        lib.kda_chunk_prefill_workspace_size.argtypes = [I64, I, I, I, I]
        lib.kda_chunk_prefill_workspace_size.restype = ctypes.c_size_t
        lib.kda_chunk_prefill.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, F, P, P, P, I, P,
                                          ctypes.c_size_t, P]
        lib.kda_chunk_prefill.restype = I
        lib.kda_chunk_prefill_gated.argtypes = [P, P, P, P, I, P, I, P, I, P, P, I, I64, I, I, I, F,
                                                P, P, P, I, P, ctypes.c_size_t, P]
        lib.kda_chunk_prefill_gated.restype = I
        lib.kda_chunk_prefill_noalloc.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, F, P, P, P,
                                                  I, P]
        lib.kda_chunk_prefill_noalloc.restype = I
        lib.kda_recurrent_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, F, P, I, P]
        lib.kda_recurrent_decode.restype = I
        lib.kda_recurrent_decode_indexed.argtypes = [P, P, P, P, P, P, I, P, I, I, I, I, I, F, P,
                                                     I, P]
        lib.kda_recurrent_decode_indexed.restype = I
        lib.kda_short_conv_qkv.argtypes = [P, P, P, P, P, P, P, I, I64, I, P, P, P, P, P, P]
        lib.kda_short_conv_qkv.restype = I
        lib.kda_short_conv_qkv_step.argtypes = [P, P, P, P, P, P, P, P, I, I, I, P, P, P, P]
        lib.kda_short_conv_qkv_step.restype = I
        lib.kda_recurrent_backward_workspace_size.argtypes = [I64, I, I, I, I]
        lib.kda_recurrent_backward_workspace_size.restype = ctypes.c_size_t
        lib.kda_recurrent_backward.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, F, P, P, I, P,
                                               P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.kda_recurrent_backward.restype = I
        lib.kda_chunk_backward_workspace_size.argtypes = [I64, I, I, I, I]
        lib.kda_chunk_backward_workspace_size.restype = ctypes.c_size_t
        lib.kda_chunk_backward.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, F, P, P, I, P,
                                           P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.kda_chunk_backward.restype = I
        lib.kda_chunk_checkpoints_size.argtypes = [I64, I, I, I, I]
        lib.kda_chunk_checkpoints_size.restype = ctypes.c_size_t
        lib.kda_chunk_prefill_checkpointed.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, F, P, P,
                                                       P, I, P, ctypes.c_size_t, P,
                                                       ctypes.c_size_t, P]
        lib.kda_chunk_prefill_checkpointed.restype = I
        lib.kda_chunk_backward_checkpointed_workspace_size.argtypes = [I64, I, I, I, I]
        lib.kda_chunk_backward_checkpointed_workspace_size.restype = ctypes.c_size_t
        lib.kda_chunk_backward_checkpointed.argtypes = [P, P, P, P, P, P, I, I64, I, I, I, F, P,
                                                        ctypes.c_size_t, P, I, P, P, P, P, P, P,
                                                        P, P, ctypes.c_size_t, P]
        lib.kda_chunk_backward_checkpointed.restype = I
        lib.kda_recurrent_decode_gated.argtypes = [P, P, P, P, I, P, I, P, I, P, P, I, P, I, I, I,
                                                   I, I, F, P, I, P]
        lib.kda_recurrent_decode_gated.restype = I
        lib.kda_gate_backward_workspace_size.argtypes = [I64, I, I]
        lib.kda_gate_backward_workspace_size.restype = ctypes.c_size_t
        lib.kda_gate_backward.argtypes = [P, I, P, I, P, I, P, P, P, P, P, P, P, I64, I, I, P,
                                          ctypes.c_size_t, P]
        lib.kda_gate_backward.restype = I
        lib.kda_page_plan.argtypes = [P, P, P, I, P, I, I, I, I, P, P, P, I64, P, P]
        lib.kda_page_plan.restype = I
        lib.kda_paged_append.argtypes = [P, P, I64, I64, P, I64, P, P]
        lib.kda_paged_append.restype = I
        lib.kda_paged_decode_workspace_size.argtypes = [I, I, I, I]
        lib.kda_paged_decode_workspace_size.restype = ctypes.c_size_t
        lib.kda_paged_decode.argtypes = [P, I64, P, P, I, P, I, I, F, P, I, P, P, ctypes.c_size_t,
                                         P]
        lib.kda_paged_decode.restype = I
        Z = ctypes.c_size_t
        lib.kda_recurrent_tree_decode.argtypes = [P, P, P, P, P, P, I, P, I, P, P, I, I64, I, I, I,
                                                  I, F, P, I, P, P]
        lib.kda_recurrent_tree_decode.restype = I
        lib.kda_recurrent_tree_commit.argtypes = [P, P, P, P, I, P, I, P, P, P, I, I64, I, I, I, I,
                                                  P]
        lib.kda_recurrent_tree_commit.restype = I
        lib.kda_short_conv_qkv_tree.argtypes = [P, P, P, P, P, P, P, P, I, P, P, I, I64, I, I, P, P,
                                                P, P]
        lib.kda_short_conv_qkv_tree.restype = I
        lib.kda_short_conv_tree_commit.argtypes = [P, P, P, P, P, I, P, P, P, I, I64, I, I, P]
        lib.kda_short_conv_tree_commit.restype = I
        lib.kda_paged_tree_decode_workspace_size.argtypes = [I, I, I, I, I]
        lib.kda_paged_tree_decode_workspace_size.restype = Z
        lib.kda_paged_tree_decode.argtypes = [P, I64, P, P, I, P, P, P, I, I64, I, I, F, P, P, P, Z,
                                              P]
        lib.kda_paged_tree_decode.restype = I
        lib.kda_paged_compact.argtypes = [P, P, I, P, P, P, P, I, I64, I, P, P]
        lib.kda_paged_compact.restype = I
        lib.kda_page_fork.argtypes = [P, P, I, P, P, I, P, I, I, I, I, P, P, P, P]
        lib.kda_page_fork.restype = I
        lib.kda_paged_copy.argtypes = [P, I, P, P]
        lib.kda_paged_copy.restype = I
        lib.kda_page_release.argtypes = [P, P, P, I, I, I, I, P, P, I, P, P]
        lib.kda_page_release.restype = I
        lib.kda_debug_check_gate_division.argtypes = [P, P]
        lib.kda_debug_check_gate_division.restype = I
        lib.kda_debug_set_wait_limit.argtypes = [I64, I64]
        lib.kda_debug_set_wait_limit.restype = I
        lib.kda_get_last_device_error.argtypes = [P]
        lib.kda_get_last_device_error.restype = I
        _lib = lib
        return lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libkda needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check(status: int, where: str):
    if status != 0:
        raise KDAError(status, where)


def kda_version() -> int:
    return load().kda_version()


def kda_status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def kda_gate_fused(f, b, A_log, alog_mode, dt_bias, g_out, beta_out, stream=None):
    N, H, K = f.shape
    st = load().kda_gate_fused(_p(f), _dtype_code(f), _p(b), _dtype_code(b) if b is not None else 0,
                               _p(A_log), int(alog_mode), _p(dt_bias), _p(g_out), _p(beta_out),
                               N, H, K, _stream(stream, f.device))
    _check(st, "kda_gate_fused")


def kda_chunk_prefill_workspace_size(N: int, B: int, H: int, K: int = 128, V: int = 128) -> int:
    return int(load().kda_chunk_prefill_workspace_size(N, B, H, K, V))


def kda_chunk_prefill(q, k, v, g, beta, cu_seqlens, scale, initial_state, final_state, o,
                      workspace, stream=None):
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().kda_chunk_prefill(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B, N, H,
                                  K, V, float(scale), _p(initial_state), _p(final_state), _p(o),
                                  _dtype_code(o), _p(workspace), ws_bytes,
                                  _stream(stream, q.device))
    _check(st, "kda_chunk_prefill")


def kda_chunk_prefill_gated(q, k, v, f, b, A_log, alog_mode, dt_bias, cu_seqlens, scale,
                            initial_state, final_state, o, workspace, stream=None):
    """Chunked prefill with the gate computed in the kernel from f, b, A_log, dt_bias."""
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().kda_chunk_prefill_gated(_p(q), _p(k), _p(v), _p(f), _dtype_code(f), _p(b),
                                        _dtype_code(b), _p(A_log), int(alog_mode), _p(dt_bias),
                                        _p(cu_seqlens), B, N, H, K, V, float(scale),
                                        _p(initial_state), _p(final_state), _p(o), _dtype_code(o),
                                        _p(workspace), ws_bytes, _stream(stream, q.device))
    _check(st, "kda_chunk_prefill_gated")


def kda_chunk_prefill_noalloc(q, k, v, g, beta, cu_seqlens, scale, initial_state, final_state, o,
                              stream=None):
    """kda_chunk_prefill with the library's built-in scratch instead of a workspace."""
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    st = load().kda_chunk_prefill_noalloc(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B,
                                          N, H, K, V, float(scale), _p(initial_state),
                                          _p(final_state), _p(o), _dtype_code(o),
                                          _stream(stream, q.device))
    _check(st, "kda_chunk_prefill_noalloc")


def kda_recurrent_decode(q, k, v, g, beta, state, scale, o, stream=None):
    B, H, K = q.shape
    V = v.shape[-1]
    st = load().kda_recurrent_decode(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(state), B, H, K, V,
                                     float(scale), _p(o), _dtype_code(o), _stream(stream, q.device))
    _check(st, "kda_recurrent_decode")


def kda_recurrent_decode_indexed(q, k, v, g, beta, state_pool, state_indices, scale, o,
                                 stream=None):
    B, H, K = q.shape
    V = v.shape[-1]
    st = load().kda_recurrent_decode_indexed(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(state_pool),
                                             _dtype_code(state_pool), _p(state_indices),
                                             state_pool.shape[0], B, H, K, V, float(scale), _p(o),
                                             _dtype_code(o), _stream(stream, q.device))
    _check(st, "kda_recurrent_decode_indexed")


def kda_short_conv_qkv(x_q, x_k, x_v, w_q, w_k, w_v, cu_seqlens, conv_state_in, conv_state_out,
                       q, k, v, stream=None):
    """x_* bf16 [N, C] (or [N, H, 128]); w_* fp32 [C, 4]; states bf16 [B, 3, 3, C]."""
    N = x_q.shape[0]
    C = w_q.shape[0]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    st = load().kda_short_conv_qkv(_p(x_q), _p(x_k), _p(x_v), _p(w_q), _p(w_k), _p(w_v),
                                   _p(cu_seqlens), B, N, C, _p(conv_state_in),
                                   _p(conv_state_out), _p(q), _p(k), _p(v),
                                   _stream(stream, x_q.device))
    _check(st, "kda_short_conv_qkv")


def kda_short_conv_qkv_step(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, state_indices, q, k,
                            v, stream=None):
    """x_* bf16 [B, C]; conv_state_pool bf16 [num_slots, 3, 3, C]; state_indices int32 [B]
    or None (slot b = sequence b)."""
    B = x_q.shape[0]
    C = w_q.shape[0]
    st = load().kda_short_conv_qkv_step(_p(x_q), _p(x_k), _p(x_v), _p(w_q), _p(w_k), _p(w_v),
                                        _p(conv_state_pool), _p(state_indices),
                                        conv_state_pool.shape[0], B, C, _p(q), _p(k), _p(v),
                                        _stream(stream, x_q.device))
    _check(st, "kda_short_conv_qkv_step")


def kda_recurrent_backward_workspace_size(N, B, H, K=128, V=128) -> int:
    return int(load().kda_recurrent_backward_workspace_size(N, B, H, K, V))


def kda_recurrent_backward(q, k, v, g, beta, cu_seqlens, scale, initial_state, dO, dS_final,
                           dq, dk, dv, dg, dbeta, dS0, workspace, stream=None):
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    st = load().kda_recurrent_backward(
        _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B, N, H, K, V, float(scale),
        _p(initial_state), _p(dO), _dtype_code(dO), _p(dS_final), _p(dq), _p(dk), _p(dv), _p(dg),
        _p(dbeta), _p(dS0), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream, q.device))
    _check(st, "kda_recurrent_backward")


def kda_chunk_backward_workspace_size(N, B, H, K=128, V=128) -> int:
    return int(load().kda_chunk_backward_workspace_size(N, B, H, K, V))


def kda_chunk_backward(q, k, v, g, beta, cu_seqlens, scale, initial_state, dO, dS_final,
                       dq, dk, dv, dg, dbeta, dS0, workspace, stream=None):
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    st = load().kda_chunk_backward(
        _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B, N, H, K, V, float(scale),
        _p(initial_state), _p(dO), _dtype_code(dO), _p(dS_final), _p(dq), _p(dk), _p(dv), _p(dg),
        _p(dbeta), _p(dS0), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream, q.device))
    _check(st, "kda_chunk_backward")


def kda_chunk_checkpoints_size(N, B, H, K=128, V=128) -> int:
    return int(load().kda_chunk_checkpoints_size(N, B, H, K, V))


def kda_chunk_prefill_checkpointed(q, k, v, g, beta, cu_seqlens, scale, initial_state,
                                   final_state, o, checkpoints, workspace, stream=None):
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().kda_chunk_prefill_checkpointed(
        _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B, N, H, K, V, float(scale),
        _p(initial_state), _p(final_state), _p(o), _dtype_code(o), _p(checkpoints),
        checkpoints.numel() * checkpoints.element_size(), _p(workspace), ws_bytes,
        _stream(stream, q.device))
    _check(st, "kda_chunk_prefill_checkpointed")


def kda_chunk_backward_checkpointed_workspace_size(N, B, H, K=128, V=128) -> int:
    return int(load().kda_chunk_backward_checkpointed_workspace_size(N, B, H, K, V))


def kda_chunk_backward_checkpointed(q, k, v, g, beta, cu_seqlens, scale, checkpoints, dO,
                                    dS_final, dq, dk, dv, dg, dbeta, dS0, workspace,
                                    stream=None):
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    st = load().kda_chunk_backward_checkpointed(
        _p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B, N, H, K, V, float(scale),
        _p(checkpoints), checkpoints.numel() * checkpoints.element_size(), _p(dO),
        _dtype_code(dO), _p(dS_final), _p(dq), _p(dk), _p(dv), _p(dg), _p(dbeta), _p(dS0),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    _check(st, "kda_chunk_backward_checkpointed")


def kda_recurrent_decode_gated(q, k, v, f, b, A_log, alog_mode, dt_bias, state_pool,
                               state_indices, scale, o, stream=None):
    """state_indices None: slot b for sequence b."""
    B, H, K = q.shape
    V = v.shape[-1]
    st = load().kda_recurrent_decode_gated(
        _p(q), _p(k), _p(v), _p(f), _dtype_code(f), _p(b), _dtype_code(b), _p(A_log),
        int(alog_mode), _p(dt_bias), _p(state_pool), _dtype_code(state_pool), _p(state_indices),
        state_pool.shape[0], B, H, K, V, float(scale), _p(o), _dtype_code(o),
        _stream(stream, q.device))
    _check(st, "kda_recurrent_decode_gated")


def kda_gate_backward_workspace_size(N, H, K) -> int:
    return int(load().kda_gate_backward_workspace_size(N, H, K))


def kda_gate_backward(f, b, A_log, alog_mode, dt_bias, dg, dbeta, df, db, dA_log, ddt_bias,
                      workspace, stream=None):
    N, H, K = f.shape
    st = load().kda_gate_backward(
        _p(f), _dtype_code(f), _p(b), KDA_FP32 if b is None else _dtype_code(b), _p(A_log),
        int(alog_mode), _p(dt_bias), _p(dg), _p(dbeta), _p(df), _p(db), _p(dA_log), _p(ddt_bias),
        N, H, K, _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream, f.device))
    _check(st, "kda_gate_backward")


class _CacheStruct(ctypes.Structure):
    """kda_paged_cache of include/kda.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class PagedCache:
    """One layer's paged key-value cache: the tensors, described once for the calls.

    k_cache, v_cache: [num_pages, page_size, heads, head_dim], bf16 or
    float8_e4m3fn, of equal strides, head_dim contiguous (pages stored head by
    head are the permuted view of [num_pages, heads, page_size, head_dim]).
    k_scale, v_scale: fp32 [heads] for an 8-bit cache, or None (1)."""

    def __init__(self, k_cache, v_cache, k_scale=None, v_scale=None):
        if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
            raise ValueError("k_cache and v_cache are [num_pages, page_size, heads, head_dim] alike")
        if k_cache.stride() != v_cache.stride() or k_cache.stride(3) != 1:
            raise ValueError("k_cache and v_cache need equal strides and a contiguous head_dim")
        if k_cache.dtype != v_cache.dtype or k_cache.device != v_cache.device:
            raise ValueError("k_cache and v_cache need one dtype and device")
        if k_cache.dtype == torch.bfloat16:
            dtype = KDA_BF16
        elif k_cache.dtype == torch.float8_e4m3fn:
            dtype = KDA_FP8_E4M3
        else:
            raise TypeError(f"unsupported cache dtype {k_cache.dtype}")
        num_pages, page_size, heads, head_dim = k_cache.shape
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or s.shape != (heads,)
                                  or s.device != k_cache.device):
                raise ValueError("a scale is fp32 [heads] on the cache's device")
        self.k_cache, self.v_cache = k_cache, v_cache
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device, self._index = k_cache.device, k_cache.get_device()
        self.num_pages, self.page_size, self.heads, self.head_dim = k_cache.shape
        self._struct = _CacheStruct(k_cache.data_ptr(), v_cache.data_ptr(), _p(k_scale),
                                    _p(v_scale), *k_cache.stride()[:3], dtype, num_pages,
                                    page_size, heads, head_dim)
        self._ref = ctypes.addressof(self._struct)


# The paged calls run once a layer and token, where the host's time counts: pointers go as
# plain integers, and the current stream's handle is asked for without a Stream object.

def _ptr(t: torch.Tensor, dtype: torch.dtype) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{dtype} tensor expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("libkda needs contiguous tensors")
    return t.data_ptr()


def _rows(t: torch.Tensor, heads: int, head_dim: int):
    """Pointer, row stride and number of bf16 [N, heads, head_dim] (or [N, heads * head_dim])
    rows, which may lie further apart than their width."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"bf16 tensor expected, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) == 3:
        ok = (shape[1] == heads and shape[2] == head_dim and strides[2] == 1
              and (heads == 1 or strides[1] == head_dim))
    else:
        ok = len(shape) == 2 and shape[1] == heads * head_dim and strides[1] == 1
    if not ok:
        raise ValueError(f"rows of {heads} x {head_dim} contiguous values expected")
    return t.data_ptr(), strides[0], shape[0]


def _elsewhere(index: int, *tensors: torch.Tensor) -> ValueError:
    """What to raise where the tensors of one call are not all on GPU `index`."""
    if index < 0:
        return ValueError("libkda needs CUDA tensors")
    return ValueError(f"tensors on cuda:{index} expected, got {[str(t.device) for t in tensors]}")


def _handle(stream, index: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def kda_page_plan(cached_lens, new_lens, free_pages, block_table, page_size, num_pages, seq_lens,
                  cu_seqlens, slot_map, pages_used, stream=None):
    """Extends block_table [B, max_pages] by pages of free_pages and maps every new token to
    its slot; writes seq_lens [B], cu_seqlens [B+1], slot_map [N] and pages_used [1]."""
    B, max_pages = block_table.shape
    if (cached_lens.numel() != B or new_lens.numel() != B or seq_lens.numel() != B
            or cu_seqlens.numel() != B + 1 or pages_used.numel() != 1):
        raise ValueError("cached_lens, new_lens, seq_lens [B], cu_seqlens [B+1], pages_used [1]")
    gpu = block_table.get_device()
    if not (0 <= gpu == cached_lens.get_device() == new_lens.get_device() == free_pages.get_device()
            == seq_lens.get_device() == cu_seqlens.get_device() == slot_map.get_device()
            == pages_used.get_device()):
        raise _elsewhere(gpu, cached_lens, new_lens, free_pages, seq_lens, cu_seqlens, slot_map,
                         pages_used)
    i32 = torch.int32
    st = (_lib or load()).kda_page_plan(
        _ptr(cached_lens, i32), _ptr(new_lens, i32), _ptr(free_pages, i32), free_pages.numel(),
        _ptr(block_table, i32), max_pages, B, page_size, num_pages, _ptr(seq_lens, i32),
        _ptr(cu_seqlens, i32), _ptr(slot_map, i32), slot_map.numel(), _ptr(pages_used, i32),
        _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_page_plan")


def kda_paged_append(k, v, slot_map, cache, stream=None):
    """k, v bf16 [N, heads, head_dim] (rows may be slices of a wider tensor); slot_map [N]."""
    N = slot_map.numel()
    kp, ks, kn = _rows(k, cache.heads, cache.head_dim)
    vp, vs, vn = _rows(v, cache.heads, cache.head_dim)
    if kn != N or vn != N:
        raise ValueError("k and v need one row per entry of slot_map")
    slots = _ptr(slot_map, torch.int32)
    gpu = cache._index
    if not (0 <= gpu == k.get_device() == v.get_device() == slot_map.get_device()):
        raise _elsewhere(gpu, k, v, slot_map)
    st = (_lib or load()).kda_paged_append(kp, vp, ks, vs, slots, N, cache._ref,
                                           _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_paged_append")


def kda_paged_decode_workspace_size(B, q_heads, kv_heads, head_dim) -> int:
    return int(load().kda_paged_decode_workspace_size(B, q_heads, kv_heads, head_dim))


def kda_paged_decode(q, cache, block_table, seq_lens, scale, o, lse, workspace, stream=None):
    """q bf16 [B, q_heads, head_dim] (rows may lie apart); o alike, bf16 or fp32; lse fp32
    [B, q_heads] or None."""
    shape = q.shape
    B, q_heads, head_dim = shape
    table_rows, max_pages = block_table.shape
    if head_dim != cache.head_dim or o.shape != shape:
        raise ValueError("q and o are [B, q_heads, head_dim] with the cache's head_dim")
    if table_rows != B or seq_lens.numel() != B:
        raise ValueError("block_table [B, max_pages] and seq_lens [B]")
    if lse is not None and lse.numel() != B * q_heads:
        raise ValueError("lse is fp32 [B, q_heads]")
    qp, qs, _ = _rows(q, q_heads, head_dim)
    o_dtype = o.dtype
    gpu = cache._index
    if not (0 <= gpu == q.get_device() == block_table.get_device() == seq_lens.get_device()
            == o.get_device() == workspace.get_device()
            == (gpu if lse is None else lse.get_device())):
        raise _elsewhere(gpu, q, block_table, seq_lens, o, workspace, *([] if lse is None else [lse]))
    st = (_lib or load()).kda_paged_decode(
        qp, qs, cache._ref, _ptr(block_table, torch.int32), max_pages,
        _ptr(seq_lens, torch.int32), B, q_heads, scale, _ptr(o, o_dtype),
        KDA_BF16 if o_dtype is torch.bfloat16 else _dtype_code(o),
        None if lse is None else _ptr(lse, torch.float32), _ptr(workspace, workspace.dtype),
        workspace.nbytes, _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_paged_decode")


def kda_debug_check_gate_division(stream=None) -> int:
    """Differing results of the gate's fast division against IEEE division
    over every operand pair of its common path (0: bit-exact)."""
    n = ctypes.c_uint64(0)
    _check(load().kda_debug_check_gate_division(ctypes.byref(n), _stream(stream)),
           "kda_debug_check_gate_division")
    return int(n.value)


def kda_debug_set_wait_limit(copy_polls: int = -1, product_polls: int = -1):
    """Test hook: bound of the chunked prefill's main-loop waits (negative = default)."""
    _check(load().kda_debug_set_wait_limit(int(copy_polls), int(product_polls)),
           "kda_debug_set_wait_limit")


def kda_get_last_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error word."""
    return int(load().kda_get_last_device_error(_stream(stream)))


# --- conveniences (allocate outputs with torch, then call the entry points) -----

def _allocates(f):
    """Lets a convenience allocate on the stream that its kernels run on.  A workspace is
    dropped while they may still run, and torch gives freed memory out again in the order of
    the stream that it was allocated on.  (So the outputs are that stream's too: whoever uses
    them on another waits for it and records that use, as for any torch tensor.)"""
    names = list(inspect.signature(f).parameters)
    place = names.index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        stream = args[place] if len(args) > place else kw.get("stream")
        if stream is None:
            return f(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            first = args[0] if args else kw[names[0]]
            stream = torch.cuda.ExternalStream(int(stream), first.device)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


@_allocates
def gate(f, b, A_log, dt_bias, alog_mode=KDA_ALOG_PER_CHANNEL, stream=None
         ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    N, H, K = f.shape
    g = torch.empty(N, H, K, dtype=torch.float32, device=f.device)
    beta = None if b is None else torch.empty(N, H, dtype=torch.float32, device=f.device)
    kda_gate_fused(f, b, A_log, alog_mode, dt_bias, g, beta, stream)
    return g, beta


@_allocates
def prefill(q, k, v, g, beta, cu_seqlens=None, scale=1.0, initial_state=None,
            o_dtype=torch.bfloat16, output_final_state=True, stream=None):
    N, H, K = q.shape
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    o = torch.empty(N, H, v.shape[-1], dtype=o_dtype, device=q.device)
    final = (torch.empty(B, H, K, v.shape[-1], dtype=torch.float32, device=q.device)
             if output_final_state else None)
    ws = torch.empty(max(kda_chunk_prefill_workspace_size(N, B, H, K, v.shape[-1]), 16),
                     dtype=torch.uint8, device=q.device)
    kda_chunk_prefill(q, k, v, g, beta, cu_seqlens, scale, initial_state, final, o, ws, stream)
    return o, final


@_allocates
def prefill_gated(q, k, v, f, b, A_log, dt_bias, alog_mode=KDA_ALOG_PER_CHANNEL, cu_seqlens=None,
                  scale=1.0, initial_state=None, o_dtype=torch.bfloat16, output_final_state=True,
                  stream=None):
    N, H, K = q.shape
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    o = torch.empty(N, H, v.shape[-1], dtype=o_dtype, device=q.device)
    final = (torch.empty(B, H, K, v.shape[-1], dtype=torch.float32, device=q.device)
             if output_final_state else None)
    ws = torch.empty(max(kda_chunk_prefill_workspace_size(N, B, H, K, v.shape[-1]), 16),
                     dtype=torch.uint8, device=q.device)
    kda_chunk_prefill_gated(q, k, v, f, b, A_log, alog_mode, dt_bias, cu_seqlens, scale,
                            initial_state, final, o, ws, stream)
    return o, final


@_allocates
def decode_indexed(q, k, v, g, beta, state_pool, state_indices, scale=1.0, o_dtype=torch.bfloat16,
                   stream=None):
    B, H, K = q.shape
    o = torch.empty(B, H, v.shape[-1], dtype=o_dtype, device=q.device)
    kda_recurrent_decode_indexed(q, k, v, g, beta, state_pool, state_indices, scale, o, stream)
    return o


@_allocates
def short_conv(x_q, x_k, x_v, w_q, w_k, w_v, cu_seqlens=None, conv_state=None,
               output_final_state=True, stream=None):
    """The pre-step on the three streams; returns (q, k, v, final conv state or None)."""
    C = w_q.shape[0]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    q, k, v = (torch.empty_like(x) for x in (x_q, x_k, x_v))
    final = (torch.empty(B, 3, 3, C, dtype=torch.bfloat16, device=x_q.device)
             if output_final_state else None)
    kda_short_conv_qkv(x_q, x_k, x_v, w_q, w_k, w_v, cu_seqlens, conv_state, final, q, k, v,
                       stream)
    return q, k, v, final


@_allocates
def short_conv_step(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, state_indices=None,
                    stream=None):
    """One token per sequence; the pool is updated in place.  Returns (q, k, v)."""
    q, k, v = (torch.empty_like(x) for x in (x_q, x_k, x_v))
    kda_short_conv_qkv_step(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, state_indices, q, k,
                            v, stream)
    return q, k, v


@_allocates
def backward(q, k, v, g, beta, dO, cu_seqlens=None, scale=1.0, initial_state=None,
             dS_final=None, want_dS0=True, stream=None):
    """Gradients of the recurrence; returns (dq, dk, dv, dg, dbeta, dS0 or None)."""
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = q.device
    dq, dk, dg = (torch.empty(N, H, K, device=dev) for _ in range(3))
    dv = torch.empty(N, H, V, device=dev)
    dbeta = torch.empty(N, H, device=dev)
    dS0 = torch.empty(B, H, K, V, device=dev) if want_dS0 else None
    ws = torch.empty(kda_recurrent_backward_workspace_size(N, B, H, K, V), dtype=torch.uint8,
                     device=dev)
    kda_recurrent_backward(q, k, v, g, beta, cu_seqlens, scale, initial_state, dO, dS_final, dq,
                           dk, dv, dg, dbeta, dS0, ws, stream)
    return dq, dk, dv, dg, dbeta, dS0


@_allocates
def backward_chunked(q, k, v, g, beta, dO, cu_seqlens=None, scale=1.0, initial_state=None,
                     dS_final=None, want_dS0=True, stream=None):
    """Gradients of the recurrence by the chunked tensor-core backward;
    returns (dq, dk, dv, dg, dbeta, dS0 or None)."""
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = q.device
    dq, dk, dg = (torch.empty(N, H, K, device=dev) for _ in range(3))
    dv = torch.empty(N, H, V, device=dev)
    dbeta = torch.empty(N, H, device=dev)
    dS0 = torch.empty(B, H, K, V, device=dev) if want_dS0 else None
    ws = torch.empty(kda_chunk_backward_workspace_size(N, B, H, K, V), dtype=torch.uint8,
                     device=dev)
    kda_chunk_backward(q, k, v, g, beta, cu_seqlens, scale, initial_state, dO, dS_final, dq, dk,
                       dv, dg, dbeta, dS0, ws, stream)
    return dq, dk, dv, dg, dbeta, dS0


@_allocates
def prefill_checkpointed(q, k, v, g, beta, cu_seqlens=None, scale=1.0, initial_state=None,
                         o_dtype=torch.bfloat16, stream=None):
    """The chunked prefill that also keeps the chunk-start states for the backward;
    returns (o, final_state, checkpoints)."""
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = q.device
    o = torch.empty(N, H, V, dtype=o_dtype, device=dev)
    final = torch.empty(B, H, K, V, dtype=torch.float32, device=dev)
    ckpt = torch.empty(kda_chunk_checkpoints_size(N, B, H, K, V), dtype=torch.uint8, device=dev)
    ws = torch.empty(max(kda_chunk_prefill_workspace_size(N, B, H, K, V), 16), dtype=torch.uint8,
                     device=dev)
    kda_chunk_prefill_checkpointed(q, k, v, g, beta, cu_seqlens, scale, initial_state, final, o,
                                   ckpt, ws, stream)
    return o, final, ckpt


@_allocates
def backward_from_checkpoints(q, k, v, g, beta, dO, checkpoints, cu_seqlens=None, scale=1.0,
                              dS_final=None, want_dS0=True, stream=None):
    """Gradients by the chunked backward from the checkpoints of prefill_checkpointed;
    returns (dq, dk, dv, dg, dbeta, dS0 or None)."""
    N, H, K = q.shape
    V = v.shape[-1]
    B = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = q.device
    dq, dk, dg = (torch.empty(N, H, K, device=dev) for _ in range(3))
    dv = torch.empty(N, H, V, device=dev)
    dbeta = torch.empty(N, H, device=dev)
    dS0 = torch.empty(B, H, K, V, device=dev) if want_dS0 else None
    ws = torch.empty(kda_chunk_backward_checkpointed_workspace_size(N, B, H, K, V),
                     dtype=torch.uint8, device=dev)
    kda_chunk_backward_checkpointed(q, k, v, g, beta, cu_seqlens, scale, checkpoints, dO,
                                    dS_final, dq, dk, dv, dg, dbeta, dS0, ws, stream)
    return dq, dk, dv, dg, dbeta, dS0


@_allocates
def decode_gated(q, k, v, f, b, A_log, dt_bias, state_pool, alog_mode=KDA_ALOG_PER_CHANNEL,
                 state_indices=None, scale=1.0, o_dtype=torch.bfloat16, stream=None):
    B, H, K = q.shape
    o = torch.empty(B, H, v.shape[-1], dtype=o_dtype, device=q.device)
    kda_recurrent_decode_gated(q, k, v, f, b, A_log, alog_mode, dt_bias, state_pool,
                               state_indices, scale, o, stream)
    return o


@_allocates
def gate_backward(f, b, A_log, dt_bias, dg, dbeta, alog_mode=KDA_ALOG_PER_CHANNEL,
                  stream=None):
    """Returns (df, db or None, dA_log, ddt_bias)."""
    N, H, K = f.shape
    dev = f.device
    df = torch.empty(N, H, K, device=dev)
    db = None if b is None else torch.empty(N, H, device=dev)
    dA = torch.empty_like(A_log)
    ddt = torch.empty(H, K, device=dev)
    ws = torch.empty(max(kda_gate_backward_workspace_size(N, H, K), 16), dtype=torch.uint8,
                     device=dev)
    kda_gate_backward(f, b, A_log, alog_mode, dt_bias, dg, dbeta, df, db, dA, ddt, ws, stream)
    return df, db, dA, ddt


@_allocates
def decode(q, k, v, g, beta, state, scale=1.0, o_dtype=torch.bfloat16, stream=None):
    B, H, K = q.shape
    o = torch.empty(B, H, v.shape[-1], dtype=o_dtype, device=q.device)
    kda_recurrent_decode(q, k, v, g, beta, state, scale, o, stream)
    return o


@_allocates
def page_plan(cached_lens, new_lens, free_pages, block_table, page_size, num_pages, num_tokens,
              stream=None):
    """Places a step's num_tokens new tokens (block_table is extended in place); returns
    (seq_lens, cu_seqlens, slot_map, pages_used)."""
    B, dev = block_table.shape[0], block_table.device
    seq_lens, cu, slots, used = (torch.empty(n, dtype=torch.int32, device=dev)
                                 for n in (B, B + 1, num_tokens, 1))
    kda_page_plan(cached_lens, new_lens, free_pages, block_table, page_size, num_pages, seq_lens,
                  cu, slots, used, stream)
    return seq_lens, cu, slots, used


@_allocates
def paged_decode(q, cache, block_table, seq_lens, scale=1.0, o_dtype=torch.bfloat16,
                 want_lse=False, stream=None):
    """Attention of one new token per sequence over the paged cache; returns (o, lse or None)."""
    B, q_heads, head_dim = q.shape
    o = torch.empty(B, q_heads, head_dim, dtype=o_dtype, device=q.device)
    lse = torch.empty(B, q_heads, device=q.device) if want_lse else None
    ws = torch.empty(max(kda_paged_decode_workspace_size(B, q_heads, cache.heads, head_dim), 16),
                     dtype=torch.uint8, device=q.device)
    kda_paged_decode(q, cache, block_table, seq_lens, scale, o, lse, ws, stream)
    return o, lse
