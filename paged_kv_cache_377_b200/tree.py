"""Speculative decoding over the paged cache: attention of drafted trees, their
masks, block tables and slots on the GPU, and the accepted path's rows.

Same names as the C ABI (include/pagedkv.h), torch tensors in. All tensors of a
call are contiguous and on the current CUDA device; the work is enqueued on
``stream`` (default: torch's current stream).
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

_loaded: Optional[ctypes.CDLL] = None
_marshal = None


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


def _calls():
    """The module that checks the arguments and makes the calls (csrc/marshal.cpp), built first if needed. Raises
    where it cannot be; no call of the other modules needs it."""
    global _marshal
    if _marshal is None:
        _lib()
        b._ensure_marshal()
        from . import _marshal as module
        _marshal = module
    return _marshal


def tree_workspace_bytes(head_dim: int) -> int:
    n = ctypes.c_size_t(0)
    b._check("pkv_tree_workspace_bytes", _lib().pkv_tree_workspace_bytes(head_dim, ctypes.byref(n)))
    return int(n.value)


def allocate_tree_workspace(head_dim: int, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace for paged_attn_tree, of any batch (its first int32 is the status word)."""
    return torch.zeros(tree_workspace_bytes(head_dim), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


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
    rc = _calls().paged_attn_tree(out, q, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask,
                                  max_query_len, scale, workspace, stream)
    if rc:
        b._check("paged_attn_tree", rc)
    return out


def paged_attn_tree_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, query_start: torch.Tensor, tree_mask: torch.Tensor,
                        max_query_len: int, scale: float, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """paged_attn_tree over e4m3 pools (uint8 [NB, bs, Hkv, D]) with fp32 per-head scales [Hkv]."""
    rc = _calls().paged_attn_tree_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                      query_start, tree_mask, max_query_len, scale, workspace, stream)
    if rc:
        b._check("paged_attn_tree_fp8", rc)
    return out


def paged_tree_mask(tree_mask: torch.Tensor, depths: torch.Tensor, parents: torch.Tensor, query_start: torch.Tensor,
                    max_query_len: int, status: torch.Tensor, stream=None) -> None:
    """tree_mask (int32 [T, words]) and depths (int32 [T]) of drafts from their parents (int32 [T]:
    an earlier draft of the same sequence, or -1 where it continues the context)."""
    rc = _calls().paged_tree_mask(tree_mask, depths, parents, query_start, max_query_len, status, stream)
    if rc:
        b._check("paged_tree_mask", rc)


def kv_tables_grow(block_tables: torch.Tensor, context_lens: torch.Tensor, new_tokens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, new_lens: torch.Tensor,
                   query_start: torch.Tensor, slot_mapping: torch.Tensor, num_free_out: torch.Tensor,
                   block_size: int, status: torch.Tensor, stream=None) -> None:
    """Room for new_tokens[s] more tokens of every sequence: blocks off the stack free_blocks
    (int32 [num_blocks], *num_free of them free) into block_tables (int32 [S, MB]), the tokens'
    slots into slot_mapping (int64, -1 behind the last), new_lens, query_start and the count left.
    new_lens may be context_lens and num_free_out may be num_free. All or nothing (see pagedkv.h)."""
    rc = _calls().kv_tables_grow(block_tables, context_lens, new_tokens, free_blocks, num_free, new_lens, query_start,
                                 slot_mapping, num_free_out, block_size, status, stream)
    if rc:
        b._check("kv_tables_grow", rc)


def kv_tables_trim(block_tables: torch.Tensor, context_lens: torch.Tensor, keep_lens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, num_free_out: torch.Tensor, block_size: int,
                   status: torch.Tensor, stream=None) -> None:
    """Gives back the blocks past keep_lens[s] of context_lens[s] tokens (0: a finished request);
    the reverse of kv_tables_grow. num_free_out may be num_free."""
    rc = _calls().kv_tables_trim(block_tables, context_lens, keep_lens, free_blocks, num_free, num_free_out, block_size,
                                 status, stream)
    if rc:
        b._check("kv_tables_trim", rc)


def kv_cache_keep(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, query_start: torch.Tensor, accepted: torch.Tensor,
                  num_accepted: torch.Tensor, new_lens: Optional[torch.Tensor], status: torch.Tensor,
                  stream=None) -> None:
    """Moves the K and V rows of each sequence's accepted drafts (accepted: int32 [S, P], rising;
    num_accepted: int32 [S]) to the places right behind its committed tokens. Pools bf16 or e4m3
    (uint8). new_lens (int32 [S] or None): committed + accepted tokens; not context_lens itself."""
    rc = _calls().kv_cache_keep(k_cache, v_cache, block_tables, context_lens, query_start, accepted, num_accepted,
                                new_lens, status, stream)
    if rc:
        b._check("kv_cache_keep", rc)
