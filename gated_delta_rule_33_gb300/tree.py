"""ctypes binding for libkda's calls over trees of drafted tokens and over shared pages
(include/kda.h): argument marshalling only, as in ``kda.py``, whose conventions hold here.

A tree is given by one word for each node, int64 [N] (the 64 bits that the C entry points
take as unsigned): bit j of a node's word is set where it sees node j of its request.
``ancestor_words`` makes the words from parents.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

from . import kda as _kda
from .kda import KDAError, _allocates, _dtype_code, _elsewhere, _handle, _ptr, _rows

KDA_TREE_MAX_NODES = 64

_I32, _I64, _F32, _B16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


def _library():
    return _kda._lib or _kda.load()


def _same_gpu(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The GPU that all of a call's tensors are on: the current one, whose kernels are launched."""
    gpu = first.get_device()
    for t in others:
        if t is not None and t.get_device() != gpu:
            raise _elsewhere(gpu, first, *(x for x in others if x is not None))
    if gpu < 0:
        raise _elsewhere(gpu)
    try:
        current = torch._C._cuda_getDevice()
    except RuntimeError:  # no driver: the library says so
        return gpu
    if gpu != current:
        raise ValueError(f"tensors on cuda:{gpu}, but the current device is cuda:{current}")
    return gpu


def _tree(cu_seqlens, ancestors, *per_request) -> Tuple[int, int]:
    """Requests and rows of a batch of trees."""
    B = cu_seqlens.numel() - 1
    for t in per_request:
        if t is not None and t.numel() != B:
            raise ValueError("cu_seqlens is [B+1], what is given for each request [B]")
    if B < 0:
        raise ValueError("cu_seqlens is [B+1]")
    return B, ancestors.numel()


def _optional(t: Optional[torch.Tensor], dtype: torch.dtype) -> Optional[int]:
    return None if t is None else _ptr(t, dtype)


def ancestor_words(parents: Sequence[int], device=None) -> torch.Tensor:
    """The words of one request's tree from its nodes' parents (-1: the context), int64 [n]:
    each node sees its ancestors and itself.  parents[i] < i."""
    words = []
    for i, p in enumerate(parents):
        if not -1 <= p < i or i >= KDA_TREE_MAX_NODES:
            raise ValueError(f"node {i} of at most {KDA_TREE_MAX_NODES}: its parent is -1 .. {i - 1}")
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64,
                        device=device)


def kda_recurrent_tree_decode(q, k, v, g, beta, state_pool, state_indices, cu_seqlens, ancestors,
                              max_nodes, scale, o, u=None, stream=None):
    """q, k, v bf16 [N, H, 128], g fp32 alike, beta fp32 [N, H]; state_pool [num_slots, H, 128,
    128] read; state_indices [B] or None; o [N, H, 128] and u (fp32, alike, or None) written."""
    B, N = _tree(cu_seqlens, ancestors, state_indices)
    slots, H, K, V = state_pool.shape
    shape = (N, H, K)
    for t in (q, k, v, g, o):
        if t.shape != shape:
            raise ValueError("q, k, v, g, o and u are [N, H, 128], N the number of words")
    if u is not None and u.shape != shape:
        raise ValueError("q, k, v, g, o and u are [N, H, 128], N the number of words")
    if beta.shape != shape[:2]:
        raise ValueError("beta is [N, H]")
    gpu = _same_gpu(q, k, v, g, beta, state_pool, state_indices, cu_seqlens, ancestors, o, u)
    st = _library().kda_recurrent_tree_decode(
        _ptr(q, _B16), _ptr(k, _B16), _ptr(v, _B16), _ptr(g, _F32), _ptr(beta, _F32),
        _ptr(state_pool, state_pool.dtype), _dtype_code(state_pool), _optional(state_indices, _I32),
        slots, _ptr(cu_seqlens, _I32), _ptr(ancestors, _I64), B, N, max_nodes, H, K, V, scale,
        _ptr(o, o.dtype), _dtype_code(o), _optional(u, _F32), _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_recurrent_tree_decode")


def kda_recurrent_tree_commit(k, g, u, state_pool, state_indices, cu_seqlens, ancestors, last,
                              max_nodes, stream=None):
    """The state after the path of node last[b] (-1: as it is), in place; k, g and u of the
    step's kda_recurrent_tree_decode."""
    B, N = _tree(cu_seqlens, ancestors, state_indices, last)
    slots, H, K, V = state_pool.shape
    for t in (k, g, u):
        if t.shape != (N, H, K):
            raise ValueError("k, g and u are [N, H, 128], N the number of words")
    gpu = _same_gpu(k, g, u, state_pool, state_indices, cu_seqlens, ancestors, last)
    st = _library().kda_recurrent_tree_commit(
        _ptr(k, _B16), _ptr(g, _F32), _ptr(u, _F32), _ptr(state_pool, state_pool.dtype),
        _dtype_code(state_pool), _optional(state_indices, _I32), slots, _ptr(cu_seqlens, _I32),
        _ptr(ancestors, _I64), _ptr(last, _I32), B, N, max_nodes, H, K, V, _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_recurrent_tree_commit")


def _conv_sizes(pool, rows, N):
    shape = pool.shape
    if len(shape) != 4 or shape[1] != 3 or shape[2] != 3:
        raise ValueError("conv_state_pool is [num_slots, 3, 3, C]")
    slots, _, _, C = shape
    for x in rows:
        if x.shape != (N, C):
            raise ValueError("x_q, x_k, x_v and the outputs are [N, C], N the number of words")
    return slots, C


def kda_short_conv_qkv_tree(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, state_indices,
                            cu_seqlens, ancestors, max_nodes, q, k, v, stream=None):
    """x, q, k, v bf16 [N, C]; w fp32 [C, 4]; conv_state_pool bf16 [num_slots, 3, 3, C], read."""
    B, N = _tree(cu_seqlens, ancestors, state_indices)
    slots, C = _conv_sizes(conv_state_pool, (x_q, x_k, x_v, q, k, v), N)
    if any(w.numel() != 4 * C for w in (w_q, w_k, w_v)):
        raise ValueError("w_q, w_k and w_v are [C, 4]")
    gpu = _same_gpu(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, state_indices, cu_seqlens,
                    ancestors, q, k, v)
    st = _library().kda_short_conv_qkv_tree(
        _ptr(x_q, _B16), _ptr(x_k, _B16), _ptr(x_v, _B16), _ptr(w_q, _F32), _ptr(w_k, _F32),
        _ptr(w_v, _F32), _ptr(conv_state_pool, _B16), _optional(state_indices, _I32), slots,
        _ptr(cu_seqlens, _I32), _ptr(ancestors, _I64), B, N, max_nodes, C, _ptr(q, _B16),
        _ptr(k, _B16), _ptr(v, _B16), _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_short_conv_qkv_tree")


def kda_short_conv_tree_commit(x_q, x_k, x_v, conv_state_pool, state_indices, cu_seqlens, ancestors,
                               last, max_nodes, stream=None):
    """The carried inputs after the path of node last[b] (-1: as they are), in place."""
    B, N = _tree(cu_seqlens, ancestors, state_indices, last)
    slots, C = _conv_sizes(conv_state_pool, (x_q, x_k, x_v), N)
    gpu = _same_gpu(x_q, x_k, x_v, conv_state_pool, state_indices, cu_seqlens, ancestors, last)
    st = _library().kda_short_conv_tree_commit(
        _ptr(x_q, _B16), _ptr(x_k, _B16), _ptr(x_v, _B16), _ptr(conv_state_pool, _B16),
        _optional(state_indices, _I32), slots, _ptr(cu_seqlens, _I32), _ptr(ancestors, _I64),
        _ptr(last, _I32), B, N, max_nodes, C, _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_short_conv_tree_commit")


def kda_paged_tree_decode_workspace_size(B, max_nodes, q_heads, kv_heads, head_dim) -> int:
    return int(_kda.load().kda_paged_tree_decode_workspace_size(B, max_nodes, q_heads, kv_heads,
                                                                head_dim))


def kda_paged_tree_decode(q, cache, block_table, seq_lens, cu_seqlens, ancestors, max_nodes, scale,
                          o, lse, workspace, stream=None):
    """q bf16 [N, q_heads, head_dim] (rows may lie apart); o bf16 alike; lse fp32 [N, q_heads] or
    None; seq_lens counts the drafted tokens."""
    B, N = _tree(cu_seqlens, ancestors, seq_lens)
    shape = q.shape
    rows, q_heads, head_dim = shape
    table_rows, max_pages = block_table.shape
    if rows != N or head_dim != cache.head_dim or o.shape != shape:
        raise ValueError("q and o are [N, q_heads, head_dim] with the cache's head_dim, N the number "
                         "of words")
    if table_rows != B:
        raise ValueError("block_table is [B, max_pages]")
    if lse is not None and lse.numel() != N * q_heads:
        raise ValueError("lse is fp32 [N, q_heads]")
    qp, qs, _ = _rows(q, q_heads, head_dim)
    gpu = _same_gpu(cache.k_cache, q, block_table, seq_lens, cu_seqlens, ancestors, o, lse, workspace)
    st = _library().kda_paged_tree_decode(
        qp, qs, cache._ref, _ptr(block_table, _I32), max_pages, _ptr(seq_lens, _I32),
        _ptr(cu_seqlens, _I32), _ptr(ancestors, _I64), B, N, max_nodes, q_heads, scale,
        _ptr(o, _B16), _optional(lse, _F32), _ptr(workspace, workspace.dtype), workspace.nbytes,
        _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_paged_tree_decode")


def kda_paged_compact(cache, block_table, seq_lens, cu_seqlens, ancestors, last, max_nodes,
                      kept_lens=None, stream=None):
    """Moves the accepted path's keys and values to where the context ends; kept_lens [B] or
    None is written."""
    B, N = _tree(cu_seqlens, ancestors, seq_lens, last, kept_lens)
    table_rows, max_pages = block_table.shape
    if table_rows != B:
        raise ValueError("block_table is [B, max_pages]")
    gpu = _same_gpu(cache.k_cache, block_table, seq_lens, cu_seqlens, ancestors, last, kept_lens)
    st = _library().kda_paged_compact(
        cache._ref, _ptr(block_table, _I32), max_pages, _ptr(seq_lens, _I32),
        _ptr(cu_seqlens, _I32), _ptr(ancestors, _I64), _ptr(last, _I32), B, N, max_nodes,
        _optional(kept_lens, _I32), _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_paged_compact")


def kda_page_fork(src, dst, seq_lens, free_pages, block_table, page_size, shares, copies, pages_used,
                  stream=None):
    """Requests dst go on from requests src: seq_lens [B], block_table [B, max_pages] and shares
    [num_pages] are updated; copies [num_forks, 3] and pages_used [1] written."""
    B, max_pages = block_table.shape
    forks = src.numel()
    if dst.numel() != forks or copies.numel() != 3 * forks or seq_lens.numel() != B \
            or pages_used.numel() != 1:
        raise ValueError("src, dst [num_forks], copies [num_forks, 3], seq_lens [B], pages_used [1]")
    gpu = _same_gpu(src, dst, seq_lens, free_pages, block_table, shares, copies, pages_used)
    st = _library().kda_page_fork(
        _ptr(src, _I32), _ptr(dst, _I32), forks, _ptr(seq_lens, _I32), _ptr(free_pages, _I32),
        free_pages.numel(), _ptr(block_table, _I32), max_pages, B, page_size, shares.numel(),
        _ptr(shares, _I32), _ptr(copies, _I32), _ptr(pages_used, _I32), _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_page_fork")


def kda_paged_copy(copies, cache, stream=None):
    """Copies pages of one layer's cache: copies int32 [num_copies, 3], each a source page, a
    destination page and a number of tokens."""
    if copies.dim() != 2 or copies.shape[1] != 3:
        raise ValueError("copies is [num_copies, 3]")
    gpu = _same_gpu(cache.k_cache, copies)
    st = _library().kda_paged_copy(_ptr(copies, _I32), copies.shape[0], cache._ref,
                                   _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_paged_copy")


def kda_page_release(seq_lens, kept_lens, block_table, page_size, shares, freed, num_freed,
                     stream=None):
    """Gives back the pages that requests of seq_lens [B] tokens no longer need for kept_lens [B];
    shares [num_pages] is updated, freed [max_freed] and num_freed [1] written.  A request that keeps
    part of a shared page must be forked before anything is appended to it."""
    B, max_pages = block_table.shape
    if seq_lens.numel() != B or kept_lens.numel() != B or num_freed.numel() != 1:
        raise ValueError("seq_lens and kept_lens [B], num_freed [1]")
    gpu = _same_gpu(seq_lens, kept_lens, block_table, shares, freed, num_freed)
    st = _library().kda_page_release(
        _ptr(seq_lens, _I32), _ptr(kept_lens, _I32), _ptr(block_table, _I32), max_pages, B,
        page_size, shares.numel(), _ptr(shares, _I32), _ptr(freed, _I32), freed.numel(),
        _ptr(num_freed, _I32), _handle(stream, gpu))
    if st:
        raise KDAError(st, "kda_page_release")


# --- conveniences (allocate outputs with torch, then call the entry points) -----

@_allocates
def recurrent_tree_decode(q, k, v, g, beta, state_pool, cu_seqlens, ancestors,
                          max_nodes=KDA_TREE_MAX_NODES, state_indices=None, scale=1.0,
                          o_dtype=torch.bfloat16, stream=None):
    """The KDA recurrence to every node of the requests' trees; returns (o, u).  Rows behind the
    last request's are not written."""
    o = torch.empty(q.shape, dtype=o_dtype, device=q.device)
    u = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    kda_recurrent_tree_decode(q, k, v, g, beta, state_pool, state_indices, cu_seqlens, ancestors,
                              max_nodes, scale, o, u, stream)
    return o, u


@_allocates
def short_conv_tree(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, cu_seqlens, ancestors,
                    max_nodes=KDA_TREE_MAX_NODES, state_indices=None, stream=None):
    """The KDA pre-step of every node; returns (q, k, v)."""
    q, k, v = (torch.empty_like(x) for x in (x_q, x_k, x_v))
    kda_short_conv_qkv_tree(x_q, x_k, x_v, w_q, w_k, w_v, conv_state_pool, state_indices, cu_seqlens,
                            ancestors, max_nodes, q, k, v, stream)
    return q, k, v


@_allocates
def paged_tree_decode(q, cache, block_table, seq_lens, cu_seqlens, ancestors,
                      max_nodes=KDA_TREE_MAX_NODES, scale=1.0, want_lse=False, stream=None):
    """Attention of every node over the paged cache; returns (o, lse or None)."""
    N, q_heads, head_dim = q.shape
    o = torch.empty(N, q_heads, head_dim, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(N, q_heads, device=q.device) if want_lse else None
    ws = torch.empty(max(kda_paged_tree_decode_workspace_size(
        block_table.shape[0], max_nodes, q_heads, cache.heads, head_dim), 16), dtype=torch.uint8,
        device=q.device)
    kda_paged_tree_decode(q, cache, block_table, seq_lens, cu_seqlens, ancestors, max_nodes, scale, o,
                          lse, ws, stream)
    return o, lse


@_allocates
def paged_compact(cache, block_table, seq_lens, cu_seqlens, ancestors, last,
                  max_nodes=KDA_TREE_MAX_NODES, stream=None):
    """Keeps the accepted paths in one layer's cache; returns kept_lens."""
    kept = torch.empty_like(seq_lens)
    kda_paged_compact(cache, block_table, seq_lens, cu_seqlens, ancestors, last, max_nodes, kept,
                      stream)
    return kept


@_allocates
def page_fork(src, dst, seq_lens, free_pages, block_table, page_size, shares, stream=None):
    """Forks requests (seq_lens, block_table and shares are updated in place); returns (copies,
    pages_used)."""
    copies = torch.empty(src.numel(), 3, dtype=torch.int32, device=block_table.device)
    used = torch.empty(1, dtype=torch.int32, device=block_table.device)
    kda_page_fork(src, dst, seq_lens, free_pages, block_table, page_size, shares, copies, used, stream)
    return copies, used


@_allocates
def page_release(seq_lens, kept_lens, block_table, page_size, shares, stream=None):
    """Gives pages back (shares is updated in place); returns (freed [num_pages], num_freed)."""
    freed = torch.empty_like(shares)
    num = torch.empty(1, dtype=torch.int32, device=shares.device)
    kda_page_release(seq_lens, kept_lens, block_table, page_size, shares, freed, num, stream)
    return freed, num
