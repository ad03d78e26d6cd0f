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

_ready = False


def _lib() -> ctypes.CDLL:
    global _ready
    lib = b.library()
    if not _ready:
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
        _ready = True
    return lib


def _one_device(*tensors: torch.Tensor) -> None:
    """Every tensor on the current CUDA device: the launch goes to its current stream."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t.device.index != here:
            raise ValueError(f"all tensors must be on the current device cuda:{here} (got {t.device})")


def tree_workspace_bytes(head_dim: int) -> int:
    n = ctypes.c_size_t(0)
    b._check("pkv_tree_workspace_bytes", _lib().pkv_tree_workspace_bytes(head_dim, ctypes.byref(n)))
    return int(n.value)


def allocate_tree_workspace(head_dim: int, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace for paged_attn_tree, of any batch (its first int32 is the status word)."""
    return torch.zeros(tree_workspace_bytes(head_dim), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _tree_sizes(out, q, k_cache, v_cache, pool_dtype, block_tables, context_lens, query_start, tree_mask, workspace):
    b._need(q, "q", torch.bfloat16, 3)
    b._need(out, "out", torch.bfloat16, 3)
    b._need(k_cache, "k_cache", pool_dtype, 4)
    b._need(v_cache, "v_cache", pool_dtype, 4)
    b._need(block_tables, "block_tables", torch.int32, 2)
    b._need(context_lens, "context_lens", torch.int32, 1)
    b._need(query_start, "query_start", torch.int32, 1)
    b._need(tree_mask, "tree_mask", torch.int32, 2)
    b._need(workspace, "workspace", torch.uint8, 1)
    _one_device(q, out, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask, workspace)
    T, Hq, D = q.shape
    NB, bs, Hkv, D2 = k_cache.shape
    S, MB = block_tables.shape
    if out.shape != q.shape or v_cache.shape != k_cache.shape or D2 != D:
        raise ValueError("shape mismatch between q/out or k_cache/v_cache")
    if context_lens.shape[0] != S or query_start.shape[0] != S + 1 or tree_mask.shape[0] != T:
        raise ValueError("context_lens needs num_seqs entries, query_start num_seqs + 1 and tree_mask num_tokens rows")
    return S, T, Hq, Hkv, D, bs, MB, NB


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
    S, T, Hq, Hkv, D, bs, MB, NB = _tree_sizes(out, q, k_cache, v_cache, torch.bfloat16, block_tables, context_lens,
                                               query_start, tree_mask, workspace)
    b._check("paged_attn_tree", _lib().paged_attn_tree(
        b._ptr(out), b._ptr(q), b._ptr(k_cache), b._ptr(v_cache), b._ptr(block_tables), b._ptr(context_lens),
        b._ptr(query_start), b._ptr(tree_mask), tree_mask.shape[1], S, T, int(max_query_len), Hq, Hkv, D, bs,
        float(scale), MB, NB, b._ptr(workspace), workspace.numel(), b._stream(stream)))
    return out


def paged_attn_tree_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, query_start: torch.Tensor, tree_mask: torch.Tensor,
                        max_query_len: int, scale: float, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """paged_attn_tree over e4m3 pools (uint8 [NB, bs, Hkv, D]) with fp32 per-head scales [Hkv]."""
    S, T, Hq, Hkv, D, bs, MB, NB = _tree_sizes(out, q, k_cache, v_cache, torch.uint8, block_tables, context_lens,
                                               query_start, tree_mask, workspace)
    b._need_scales(k_scale, v_scale, Hkv)
    _one_device(k_scale, v_scale)
    b._check("paged_attn_tree_fp8", _lib().paged_attn_tree_fp8(
        b._ptr(out), b._ptr(q), b._ptr(k_cache), b._ptr(v_cache), b._ptr(k_scale), b._ptr(v_scale),
        b._ptr(block_tables), b._ptr(context_lens), b._ptr(query_start), b._ptr(tree_mask), tree_mask.shape[1], S, T,
        int(max_query_len), Hq, Hkv, D, bs, float(scale), MB, NB, b._ptr(workspace), workspace.numel(),
        b._stream(stream)))
    return out


def paged_tree_mask(tree_mask: torch.Tensor, depths: torch.Tensor, parents: torch.Tensor, query_start: torch.Tensor,
                    max_query_len: int, status: torch.Tensor, stream=None) -> None:
    """tree_mask (int32 [T, words]) and depths (int32 [T]) of drafts from their parents (int32 [T]:
    an earlier draft of the same sequence, or -1 where it continues the context)."""
    b._need(tree_mask, "tree_mask", torch.int32, 2)
    b._need(depths, "depths", torch.int32, 1)
    b._need(parents, "parents", torch.int32, 1)
    b._need(query_start, "query_start", torch.int32, 1)
    b._need(status, "status", torch.int32, 1)
    _one_device(tree_mask, depths, parents, query_start, status)
    T = parents.shape[0]
    if tree_mask.shape[0] != T or depths.shape[0] != T or query_start.shape[0] < 1:
        raise ValueError("tree_mask and depths need a row per token, query_start num_seqs + 1 entries")
    b._check("paged_tree_mask", _lib().paged_tree_mask(
        b._ptr(tree_mask), b._ptr(depths), b._ptr(parents), b._ptr(query_start), query_start.shape[0] - 1, T,
        int(max_query_len), tree_mask.shape[1], b._ptr(status), b._stream(stream)))


def kv_tables_grow(block_tables: torch.Tensor, context_lens: torch.Tensor, new_tokens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, new_lens: torch.Tensor,
                   query_start: torch.Tensor, slot_mapping: torch.Tensor, num_free_out: torch.Tensor,
                   block_size: int, status: torch.Tensor, stream=None) -> None:
    """Room for new_tokens[s] more tokens of every sequence: blocks off the stack free_blocks
    (int32 [num_blocks], *num_free of them free) into block_tables (int32 [S, MB]), the tokens'
    slots into slot_mapping (int64, -1 behind the last), new_lens, query_start and the count left.
    new_lens may be context_lens and num_free_out may be num_free. All or nothing (see pagedkv.h)."""
    b._need(block_tables, "block_tables", torch.int32, 2)
    b._need(slot_mapping, "slot_mapping", torch.int64, 1)
    for t, name in ((context_lens, "context_lens"), (new_tokens, "new_tokens"), (free_blocks, "free_blocks"),
                    (num_free, "num_free"), (new_lens, "new_lens"), (query_start, "query_start"),
                    (num_free_out, "num_free_out"), (status, "status")):
        b._need(t, name, torch.int32, 1)
    _one_device(block_tables, slot_mapping, context_lens, new_tokens, free_blocks, num_free, new_lens, query_start,
                num_free_out, status)
    S, MB = block_tables.shape
    if context_lens.shape[0] != S or new_tokens.shape[0] != S or new_lens.shape[0] != S or \
            query_start.shape[0] != S + 1 or num_free.shape[0] != 1 or num_free_out.shape[0] != 1:
        raise ValueError("context_lens, new_tokens and new_lens need num_seqs entries, query_start num_seqs + 1, "
                         "num_free and num_free_out one")
    b._check("kv_tables_grow", _lib().kv_tables_grow(
        b._ptr(block_tables), b._ptr(context_lens), b._ptr(new_tokens), b._ptr(free_blocks), b._ptr(num_free),
        b._ptr(new_lens), b._ptr(query_start), b._ptr(slot_mapping), b._ptr(num_free_out), S, slot_mapping.shape[0],
        MB, int(block_size), free_blocks.shape[0], b._ptr(status), b._stream(stream)))


def kv_tables_trim(block_tables: torch.Tensor, context_lens: torch.Tensor, keep_lens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, num_free_out: torch.Tensor, block_size: int,
                   status: torch.Tensor, stream=None) -> None:
    """Gives back the blocks past keep_lens[s] of context_lens[s] tokens (0: a finished request);
    the reverse of kv_tables_grow. num_free_out may be num_free."""
    b._need(block_tables, "block_tables", torch.int32, 2)
    for t, name in ((context_lens, "context_lens"), (keep_lens, "keep_lens"), (free_blocks, "free_blocks"),
                    (num_free, "num_free"), (num_free_out, "num_free_out"), (status, "status")):
        b._need(t, name, torch.int32, 1)
    _one_device(block_tables, context_lens, keep_lens, free_blocks, num_free, num_free_out, status)
    S, MB = block_tables.shape
    if context_lens.shape[0] != S or keep_lens.shape[0] != S or num_free.shape[0] != 1 or num_free_out.shape[0] != 1:
        raise ValueError("context_lens and keep_lens need num_seqs entries, num_free and num_free_out one")
    b._check("kv_tables_trim", _lib().kv_tables_trim(
        b._ptr(block_tables), b._ptr(context_lens), b._ptr(keep_lens), b._ptr(free_blocks), b._ptr(num_free),
        b._ptr(num_free_out), S, MB, int(block_size), free_blocks.shape[0], b._ptr(status), b._stream(stream)))


def kv_cache_keep(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, query_start: torch.Tensor, accepted: torch.Tensor,
                  num_accepted: torch.Tensor, new_lens: Optional[torch.Tensor], status: torch.Tensor,
                  stream=None) -> None:
    """Moves the K and V rows of each sequence's accepted drafts (accepted: int32 [S, P], rising;
    num_accepted: int32 [S]) to the places right behind its committed tokens. Pools bf16 or e4m3
    (uint8). new_lens (int32 [S] or None): committed + accepted tokens; not context_lens itself."""
    pool = k_cache.dtype if isinstance(k_cache, torch.Tensor) and k_cache.dtype == torch.uint8 else torch.bfloat16
    b._need(k_cache, "k_cache", pool, 4)
    b._need(v_cache, "v_cache", pool, 4)
    b._need(block_tables, "block_tables", torch.int32, 2)
    b._need(accepted, "accepted", torch.int32, 2)
    for t, name in ((context_lens, "context_lens"), (query_start, "query_start"), (num_accepted, "num_accepted"),
                    (status, "status")):
        b._need(t, name, torch.int32, 1)
    _one_device(k_cache, v_cache, block_tables, accepted, context_lens, query_start, num_accepted, status)
    S, MB = block_tables.shape
    NB, bs, Hkv, D = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between k_cache and v_cache")
    if context_lens.shape[0] != S or query_start.shape[0] != S + 1 or accepted.shape[0] != S or \
            num_accepted.shape[0] != S:
        raise ValueError("context_lens, accepted and num_accepted need num_seqs rows, query_start num_seqs + 1")
    if new_lens is not None:
        b._need(new_lens, "new_lens", torch.int32, 1)
        _one_device(new_lens)
        if new_lens.shape[0] != S:
            raise ValueError("new_lens needs num_seqs entries")
    b._check("kv_cache_keep", _lib().kv_cache_keep(
        b._ptr(k_cache), b._ptr(v_cache), b._ptr(block_tables), b._ptr(context_lens), b._ptr(query_start),
        b._ptr(accepted), b._ptr(num_accepted), b._ptr(new_lens), S, accepted.shape[1], Hkv, D,
        k_cache.element_size(), bs, MB, NB, b._ptr(status), b._stream(stream)))
