"""Speculative decoding over the paged cache: attention of drafted trees, their
masks, block tables and slots on the GPU, and the accepted path's rows.

Same names as the C ABI (include/pagedkv.h), torch tensors in; only the
arguments are marshalled here.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _binding as b

PKV_STATUS_BAD_TREE = 32
PKV_STATUS_OUT_OF_BLOCKS = 64
PKV_STATUS_OUT_OF_SLOTS = 128
PKV_MAX_TREE_TOKENS = 4096

_BF16, _U8, _I32, _I64, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32
_loaded: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _loaded
    if _loaded is None:
        lib = b.library()
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sizes = [I] * 8 + [F, I, I, P, Z, P]
        for name, args in (("pkv_tree_workspace_bytes", [I, ctypes.POINTER(Z)]),
                           ("paged_attn_tree", [P] * 8 + sizes),
                           ("paged_attn_tree_fp8", [P] * 10 + sizes),
                           ("paged_tree_mask", [P] * 4 + [I] * 4 + [P, P]),
                           ("kv_tables_grow", [P] * 9 + [I] * 5 + [P, P]),
                           ("kv_tables_trim", [P] * 6 + [I] * 4 + [P, P]),
                           ("kv_cache_keep", [P] * 8 + [I] * 8 + [P, P])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = I, args
        _loaded = lib
    return _loaded


def _pointers(*specs):
    """Device pointers of (tensor, name, dtype, dimensions): contiguous, and all on the current CUDA device, where the
    launch goes. The small calls of a step are as long as their arguments take to check, hence the one loop."""
    first = specs[0][0]
    here = first.get_device() if isinstance(first, torch.Tensor) else -1
    out = []
    for t, name, dtype, ndim in specs:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()
                and t.get_device() == here >= 0):
            b._need(t, name, dtype, ndim)
            raise ValueError(f"all tensors must be on one device ({name} is on {t.device})")
        out.append(t.data_ptr())
    if here != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{here}, not on the current device cuda:{torch.cuda.current_device()}")
    return out


# the current stream's handle, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream, device: int):
    return _raw_stream(device) if stream is None else b._stream(stream)


def tree_workspace_bytes(head_dim: int) -> int:
    n = ctypes.c_size_t(0)
    b._check("pkv_tree_workspace_bytes", _lib().pkv_tree_workspace_bytes(head_dim, ctypes.byref(n)))
    return int(n.value)


def allocate_tree_workspace(head_dim: int, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace for paged_attn_tree, of any batch (its first int32 is the status word)."""
    return torch.zeros(tree_workspace_bytes(head_dim), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _tree(name, out, q, k_cache, v_cache, pool, scales, block_tables, context_lens, query_start, tree_mask,
          max_query_len, scale, workspace, stream):
    ptrs = _pointers((out, "out", _BF16, 3), (q, "q", _BF16, 3), (k_cache, "k_cache", pool, 4),
                     (v_cache, "v_cache", pool, 4), *scales, (block_tables, "block_tables", _I32, 2),
                     (context_lens, "context_lens", _I32, 1), (query_start, "query_start", _I32, 1),
                     (tree_mask, "tree_mask", _I32, 2), (workspace, "workspace", _U8, 1))
    T, Hq, D = q.shape
    NB, bs, Hkv, D2 = k_cache.shape
    S, MB = block_tables.shape
    rows, words = tree_mask.shape
    if out.shape != q.shape or v_cache.shape != k_cache.shape or D2 != D:
        raise ValueError("shape mismatch between q/out or k_cache/v_cache")
    if context_lens.shape[0] != S or query_start.shape[0] != S + 1 or rows != T:
        raise ValueError("context_lens needs num_seqs entries, query_start num_seqs + 1 and tree_mask num_tokens rows")
    for t, what, _, _ in scales:
        if t.shape[0] != Hkv:
            raise ValueError("k_scale and v_scale must have num_kv_heads entries")
    b._check(name, getattr(_lib(), name)(
        *ptrs[:-1], words, S, T, max_query_len, Hq, Hkv, D, bs, scale, MB, NB, ptrs[-1], workspace.shape[0],
        _stream(stream, q.get_device())))
    return out


def paged_attn_tree(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor,
                    tree_mask: torch.Tensor, max_query_len: int, scale: float, workspace: torch.Tensor,
                    stream=None) -> torch.Tensor:
    """Attention of drafted tokens over the cache and the drafts their mask rows name.

    q, out: bf16 [T, Hq, D], the drafts of sequence s in rows query_start[s] ..
    query_start[s+1]-1, which are the last tokens of its context;
    tree_mask: int32 [T, words], bit j = draft j of the sequence is seen (paged_tree_mask);
    workspace: uint8 from allocate_tree_workspace(). A row that sees nothing gives zeros.
    """
    return _tree("paged_attn_tree", out, q, k_cache, v_cache, _BF16, (), block_tables, context_lens, query_start,
                 tree_mask, max_query_len, scale, workspace, stream)


def paged_attn_tree_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, query_start: torch.Tensor, tree_mask: torch.Tensor,
                        max_query_len: int, scale: float, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """paged_attn_tree over e4m3 pools (uint8 [NB, bs, Hkv, D]) with fp32 per-head scales [Hkv]."""
    return _tree("paged_attn_tree_fp8", out, q, k_cache, v_cache, _U8,
                 ((k_scale, "k_scale", _F32, 1), (v_scale, "v_scale", _F32, 1)), block_tables, context_lens,
                 query_start, tree_mask, max_query_len, scale, workspace, stream)


def paged_tree_mask(tree_mask: torch.Tensor, depths: torch.Tensor, parents: torch.Tensor, query_start: torch.Tensor,
                    max_query_len: int, status: torch.Tensor, stream=None) -> None:
    """tree_mask (int32 [T, words]) and depths (int32 [T]) of drafts from their parents (int32 [T]:
    an earlier draft of the same sequence, or -1 where it continues the context)."""
    pm, pd, pp, pq, ps = _pointers((tree_mask, "tree_mask", _I32, 2), (depths, "depths", _I32, 1),
                                   (parents, "parents", _I32, 1), (query_start, "query_start", _I32, 1),
                                   (status, "status", _I32, 1))
    T, S = parents.shape[0], query_start.shape[0] - 1
    rows, words = tree_mask.shape
    if rows != T or depths.shape[0] != T or S < 0 or status.shape[0] < 1:
        raise ValueError("tree_mask and depths need a row per token, query_start num_seqs + 1 entries, status one")
    b._check("paged_tree_mask", _lib().paged_tree_mask(pm, pd, pp, pq, S, T, max_query_len, words, ps,
                                                       _stream(stream, parents.get_device())))


def kv_tables_grow(block_tables: torch.Tensor, context_lens: torch.Tensor, new_tokens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, new_lens: torch.Tensor,
                   query_start: torch.Tensor, slot_mapping: torch.Tensor, num_free_out: torch.Tensor,
                   block_size: int, status: torch.Tensor, stream=None) -> None:
    """Room for new_tokens[s] more tokens of every sequence: blocks off the stack free_blocks
    (int32 [num_blocks], *num_free of them free) into block_tables (int32 [S, MB]), the tokens'
    slots into slot_mapping (int64, -1 behind the last), new_lens, query_start and the count left.
    new_lens may be context_lens and num_free_out may be num_free. All or nothing (see pagedkv.h)."""
    ptrs = _pointers((block_tables, "block_tables", _I32, 2), (context_lens, "context_lens", _I32, 1),
                     (new_tokens, "new_tokens", _I32, 1), (free_blocks, "free_blocks", _I32, 1),
                     (num_free, "num_free", _I32, 1), (new_lens, "new_lens", _I32, 1),
                     (query_start, "query_start", _I32, 1), (slot_mapping, "slot_mapping", _I64, 1),
                     (num_free_out, "num_free_out", _I32, 1), (status, "status", _I32, 1))
    S, MB = block_tables.shape
    if context_lens.shape[0] != S or new_tokens.shape[0] != S or new_lens.shape[0] != S or \
            query_start.shape[0] != S + 1 or num_free.shape[0] != 1 or num_free_out.shape[0] != 1 or \
            status.shape[0] < 1:
        raise ValueError("context_lens, new_tokens and new_lens need num_seqs entries, query_start num_seqs + 1, "
                         "num_free, num_free_out and status one")
    b._check("kv_tables_grow", _lib().kv_tables_grow(
        *ptrs[:-1], S, slot_mapping.shape[0], MB, block_size, free_blocks.shape[0], ptrs[-1],
        _stream(stream, block_tables.get_device())))


def kv_tables_trim(block_tables: torch.Tensor, context_lens: torch.Tensor, keep_lens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, num_free_out: torch.Tensor, block_size: int,
                   status: torch.Tensor, stream=None) -> None:
    """Gives back the blocks past keep_lens[s] of context_lens[s] tokens (0: a finished request);
    the reverse of kv_tables_grow. num_free_out may be num_free."""
    ptrs = _pointers((block_tables, "block_tables", _I32, 2), (context_lens, "context_lens", _I32, 1),
                     (keep_lens, "keep_lens", _I32, 1), (free_blocks, "free_blocks", _I32, 1),
                     (num_free, "num_free", _I32, 1), (num_free_out, "num_free_out", _I32, 1),
                     (status, "status", _I32, 1))
    S, MB = block_tables.shape
    if context_lens.shape[0] != S or keep_lens.shape[0] != S or num_free.shape[0] != 1 or \
            num_free_out.shape[0] != 1 or status.shape[0] < 1:
        raise ValueError("context_lens and keep_lens need num_seqs entries, num_free, num_free_out and status one")
    b._check("kv_tables_trim", _lib().kv_tables_trim(*ptrs[:-1], S, MB, block_size, free_blocks.shape[0], ptrs[-1],
                                                     _stream(stream, block_tables.get_device())))


def kv_cache_keep(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, query_start: torch.Tensor, accepted: torch.Tensor,
                  num_accepted: torch.Tensor, new_lens: Optional[torch.Tensor], status: torch.Tensor,
                  stream=None) -> None:
    """Moves the K and V rows of each sequence's accepted drafts (accepted: int32 [S, P], rising;
    num_accepted: int32 [S]) to the places right behind its committed tokens. Pools bf16 or e4m3
    (uint8). new_lens (int32 [S] or None): committed + accepted tokens; not context_lens itself."""
    pool = _U8 if isinstance(k_cache, torch.Tensor) and k_cache.dtype is _U8 else _BF16
    last = ((new_lens, "new_lens", _I32, 1),) if new_lens is not None else ()
    ptrs = _pointers((k_cache, "k_cache", pool, 4), (v_cache, "v_cache", pool, 4),
                     (block_tables, "block_tables", _I32, 2), (context_lens, "context_lens", _I32, 1),
                     (query_start, "query_start", _I32, 1), (accepted, "accepted", _I32, 2),
                     (num_accepted, "num_accepted", _I32, 1), (status, "status", _I32, 1), *last)
    S, MB = block_tables.shape
    NB, bs, Hkv, D = k_cache.shape
    A, P = accepted.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between k_cache and v_cache")
    if context_lens.shape[0] != S or query_start.shape[0] != S + 1 or A != S or num_accepted.shape[0] != S or \
            status.shape[0] < 1 or (new_lens is not None and new_lens.shape[0] != S):
        raise ValueError("context_lens, accepted, num_accepted and new_lens need num_seqs rows, query_start "
                         "num_seqs + 1, status one")
    b._check("kv_cache_keep", _lib().kv_cache_keep(
        *ptrs[:7], ptrs[8] if last else None, S, P, Hkv, D, 1 if pool is _U8 else 2, bs, MB, NB, ptrs[7],
        _stream(stream, k_cache.get_device())))
