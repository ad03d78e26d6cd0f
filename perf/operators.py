"""Cases for the speculative-decoding operators of the paged KV cache.

A step that verifies a tree of drafted tokens per sequence runs: block tables
and slots for the drafts (``kv_tables_grow``), the tree's visibility mask
(``paged_tree_mask``), attention of every drafted token over the committed
cache and its own ancestors (``paged_attn_tree``, ``paged_attn_tree_fp8``),
then the accepted path's rows moved together (``kv_cache_keep``) and the
blocks that fell empty given back (``kv_tables_trim``).

``run`` computes each of them from elementary torch operations, or with
``own`` set through the package's entry points; ``exact`` computes them in 64
bits, sequence by sequence.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def _attn(name, seqs, q_heads, kv_heads, head_dim, block_size, ctx_lo, ctx_hi, skew, nodes_lo, nodes_hi, fp8=False):
    case = dict(op="attn", seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
                ctx_lo=ctx_lo, ctx_hi=ctx_hi, skew=skew, nodes_lo=nodes_lo, nodes_hi=nodes_hi, fp8=fp8)
    return dict(name=name, **case) if name else case


def _mask(name, seqs, nodes_lo, nodes_hi, chain):
    case = dict(op="mask", seqs=seqs, nodes_lo=nodes_lo, nodes_hi=nodes_hi, chain=chain)
    return dict(name=name, **case) if name else case


def _grow(name, seqs, block_size, ctx_lo, ctx_hi, new_lo, new_hi):
    case = dict(op="grow", seqs=seqs, block_size=block_size, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo,
                new_hi=new_hi)
    return dict(name=name, **case) if name else case


def _trim(name, seqs, block_size, ctx_lo, ctx_hi, finished, drop_hi):
    case = dict(op="trim", seqs=seqs, block_size=block_size, ctx_lo=ctx_lo, ctx_hi=ctx_hi, finished=finished,
                drop_hi=drop_hi)
    return dict(name=name, **case) if name else case


def _keep(name, seqs, kv_heads, head_dim, block_size, ctx_lo, ctx_hi, nodes_lo, nodes_hi, accept_hi, fp8):
    case = dict(op="keep", seqs=seqs, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, ctx_lo=ctx_lo,
                ctx_hi=ctx_hi, nodes_lo=nodes_lo, nodes_hi=nodes_hi, accept_hi=accept_hi, fp8=fp8)
    return dict(name=name, **case) if name else case


def listed():
    return [
        # the smallest step: four short chats with a handful of drafts each; latency is all of it
        _attn("tree_tiny", 4, 2, 1, 64, 16, 1, 33, False, 1, 7),
        # a serving batch of Llama-3-8B heads verifying wide trees: 256 query rows per kv head
        _attn("tree_llama_wide", 64, 32, 8, 128, 16, 128, 4096, False, 48, 64),
        # few long documents, small ragged trees, seven query heads per kv head: the context has to be split
        _attn("tree_long_group7", 8, 28, 4, 128, 32, 4096, 32768, True, 5, 26),
        # the serving batch on an e4m3 cache, chains and small trees
        _attn("tree_llama_e4m3", 64, 32, 8, 128, 16, 128, 4096, False, 4, 16, fp8=True),
        # visibility of a serving batch's trees, and of one request's longest single chain
        _mask("mask_batch", 256, 33, 64, False),
        _mask("mask_chain", 2, 250, 256, True),
        # a plain decode step of a full batch: one token each, a block now and then
        _grow("grow_decode", 256, 16, 128, 4096, 1, 1),
        # admission of many prompts at once beside running requests
        _grow("grow_admit", 1000, 16, 0, 1024, 1, 512),
        # rejected drafts given back after a verified step
        _trim("trim_drafts", 256, 16, 128, 4096, 0.0, 63),
        # a drain: half the requests end and return all they held
        _trim("trim_finished", 1000, 32, 1, 4096, 0.5, 31),
        # accepted paths moved together, bf16 rows of eight heads
        _keep("keep_llama", 64, 8, 128, 16, 128, 2048, 48, 64, 12, False),
        # the same in a large batch on e4m3 rows
        _keep("keep_e4m3", 256, 8, 128, 32, 16, 512, 16, 64, 16, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


_HEADS = [(2, 1, 64), (12, 12, 64), (32, 8, 128), (28, 4, 128), (24, 8, 128), (16, 16, 128), (40, 8, 64)]


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn_fp8", "attn_fp8", "mask", "grow", "trim", "keep", "keep"])
    bs = rng.choice([16, 32])
    if op in ("attn", "attn_fp8"):
        hq, hkv, d = rng.choice(_HEADS)
        nodes = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 16, 32768)
        seqs = _log_int(rng, 1, max(1, min(64, 64 * 4096 // ctx)))
        return _attn(None, seqs, hq, hkv, d, bs, rng.randint(0, ctx // 2), ctx, rng.random() < 0.4,
                     rng.randint(1, nodes), nodes, op == "attn_fp8")
    if op == "mask":
        nodes = _log_int(rng, 1, 256)
        return _mask(None, _log_int(rng, 1, 512), rng.randint(1, nodes), nodes, rng.random() < 0.2)
    if op == "grow":
        ctx, new = _log_int(rng, 16, 8192), _log_int(rng, 1, 512)
        return _grow(None, _log_int(rng, 1, 1500), bs, rng.randint(0, ctx // 2), ctx, rng.randint(0, new // 2), new)
    if op == "trim":
        ctx = _log_int(rng, 64, 8192)
        return _trim(None, _log_int(rng, 1, 1500), bs, rng.randint(0, ctx // 2), ctx, rng.choice([0.0, 0.1, 0.5]),
                     rng.randint(1, 63))
    nodes, ctx = _log_int(rng, 2, 64), _log_int(rng, 16, 1024)
    _, hkv, d = rng.choice(_HEADS)
    return _keep(None, _log_int(rng, 1, 256), hkv, d, bs, rng.randint(0, ctx // 2), ctx, rng.randint(1, nodes), nodes,
                 rng.randint(1, 16), rng.random() < 0.4)


# ---------------------------------------------------------------- inputs

def _lengths(case, rng):
    """Committed tokens of each sequence: uniform, or spread over the logarithm with one at the top."""
    lo, hi, n = case["ctx_lo"], case["ctx_hi"], case["seqs"]
    if case.get("skew"):
        x = np.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1), size=n)).astype(np.int64).clip(lo, hi)
        x[rng.integers(n)] = hi
        return x
    return rng.integers(lo, hi + 1, size=n)


def _ragged(lo, hi, n, rng):
    """n whole numbers of [lo, hi] whose sum is the middle of the range: a step's token budget."""
    x = rng.integers(lo, hi + 1, size=n)
    left = n * (lo + hi) // 2 - int(x.sum())
    while left:
        room = np.flatnonzero(x < hi if left > 0 else x > lo)
        some = rng.permutation(room)[:abs(left)]
        x[some] += 1 if left > 0 else -1
        left -= len(some) if left > 0 else -len(some)
    return x


def _parents(nodes, chain, rng):
    """Per sequence, the parent of each node (an earlier node, or -1)."""
    out = []
    for n in nodes:
        i = np.arange(n)
        if chain:
            out.append(i - 1)
        else:  # wide at the top, thinner below, as drafts ranked by probability are
            out.append(np.floor((i + 1) * rng.random(n) ** 1.5).astype(np.int64) - 1)
    return out


def _ancestors(parents):
    """Boolean [n, n]: node i sees node j (its ancestors and itself)."""
    n = len(parents)
    a = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            a[i] = a[p]
        a[i, i] = True
    return a


def _pack_rows(bools, words):
    pad = np.zeros((bools.shape[0], words * 32), dtype=bool)
    pad[:, :bools.shape[1]] = bools
    return np.packbits(pad, axis=1, bitorder="little").view(np.int32)


def _tables(lens, bs, width, num_blocks, rng):
    """Random distinct physical blocks; returns (tables padded with -1, the unused blocks in random order)."""
    need = -(-lens // bs)
    perm = rng.permutation(num_blocks).astype(np.int32)
    t = np.full((len(lens), width), -1, dtype=np.int32)
    cols = np.arange(width)[None, :] < need[:, None]
    t[cols] = perm[:int(need.sum())]
    return t, perm[int(need.sum()):]


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _codes(shape, gen):
    """e4m3 codes of both signs, magnitudes 2^-3 .. 30."""
    sign = torch.randint(0, 2, shape, generator=gen, device=DEV, dtype=torch.uint8)
    return (sign << 7) | torch.randint(32, 96, shape, generator=gen, device=DEV, dtype=torch.uint8)


def _pools(case, num_blocks, gen):
    shape = (num_blocks, case["block_size"], case["kv_heads"], case["head_dim"])
    if case["fp8"]:
        return _codes(shape, gen), _codes(shape, gen)
    return tuple(torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))


def _attn_sizes(case, rng):
    base = _lengths(case, rng)
    return base, _ragged(case["nodes_lo"], case["nodes_hi"], case["seqs"], rng)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return _PREPARE[case["op"]](case, rng, gen)


def _prepare_attn(case, rng, gen):
    base, nodes = _attn_sizes(case, rng)
    bs, hq, hkv, d = case["block_size"], case["q_heads"], case["kv_heads"], case["head_dim"]
    lens = base + nodes
    width = -(-(case["ctx_hi"] + case["nodes_hi"]) // bs)
    num_blocks = case["seqs"] * width + 8
    tables, _ = _tables(lens, bs, width, num_blocks, rng)
    words = -(-case["nodes_hi"] // 32)
    mask = np.concatenate([_pack_rows(_ancestors(p), words) for p in _parents(nodes, False, rng)])
    total = int(nodes.sum())
    kc, vc = _pools(case, num_blocks, gen)
    q = torch.randn(total, hq, d, generator=gen, device=DEV, dtype=torch.bfloat16)
    s = dict(case=case, q=q, out=torch.empty_like(q), k_cache=kc, v_cache=vc, block_tables=_dev(tables),
             context_lens=_dev(lens), query_start=_dev(np.concatenate([[0], np.cumsum(nodes)])),
             tree_mask=_dev(mask), max_query_len=case["nodes_hi"], scale=1.0 / math.sqrt(d))
    if case["fp8"]:
        h = torch.arange(hkv, device=DEV, dtype=torch.float32)
        s["k_scale"], s["v_scale"] = 2.0 ** -4 * (1 + h / hkv), 2.0 ** -4 * (1 + h / (2 * hkv))
    return s


def _prepare_mask(case, rng, gen):
    nodes = _ragged(case["nodes_lo"], case["nodes_hi"], case["seqs"], rng)
    words = -(-case["nodes_hi"] // 32)
    total = int(nodes.sum())
    return dict(case=case, parents=_dev(np.concatenate(_parents(nodes, case["chain"], rng))),
                query_start=_dev(np.concatenate([[0], np.cumsum(nodes)])),
                tree_mask=torch.empty(total, words, dtype=torch.int32, device=DEV),
                depths=torch.empty(total, dtype=torch.int32, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV), max_query_len=case["nodes_hi"])


def _grow_sizes(case, rng):
    return _lengths(case, rng), _ragged(case["new_lo"], case["new_hi"], case["seqs"], rng)


def _prepare_grow(case, rng, gen):
    lens, new = _grow_sizes(case, rng)
    bs = case["block_size"]
    width = -(-(case["ctx_hi"] + case["new_hi"]) // bs)
    num_blocks = case["seqs"] * width + 16
    tables, free = _tables(lens, bs, width, num_blocks, rng)
    stack = np.full(num_blocks, -1, dtype=np.int32)
    stack[:len(free)] = free
    slots = int(new.sum()) + 5 * case["seqs"] // 4  # a step's fixed token budget: some of it stays unused
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, block_tables=_dev(tables), context_lens=_dev(lens), new_tokens=_dev(new),
                free_blocks=_dev(stack), num_free=torch.full((1,), len(free), **i32),
                new_lens=torch.empty(case["seqs"], **i32), query_start=torch.empty(case["seqs"] + 1, **i32),
                slot_mapping=torch.empty(slots, dtype=torch.int64, device=DEV), num_free_out=torch.empty(1, **i32),
                status=torch.zeros(1, **i32))


def _trim_sizes(case, rng):
    lens = _lengths(case, rng)
    keep = np.maximum(lens - rng.integers(0, case["drop_hi"] + 1, size=case["seqs"]), 0)
    keep[rng.random(case["seqs"]) < case["finished"]] = 0
    return lens, keep


def _prepare_trim(case, rng, gen):
    lens, keep = _trim_sizes(case, rng)
    bs = case["block_size"]
    width = -(-case["ctx_hi"] // bs)
    num_blocks = case["seqs"] * width + 16
    tables, free = _tables(lens, bs, width, num_blocks, rng)
    stack = np.full(num_blocks, -1, dtype=np.int32)
    stack[:len(free)] = free
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, block_tables=_dev(tables), context_lens=_dev(lens), keep_lens=_dev(keep),
                free_blocks=_dev(stack), num_free=torch.full((1,), len(free), **i32),
                num_free_out=torch.empty(1, **i32), status=torch.zeros(1, **i32))


def _keep_sizes(case, rng):
    base, nodes = _attn_sizes(case, rng)
    return base, nodes, np.minimum(nodes, rng.integers(0, case["accept_hi"] + 1, size=case["seqs"]))


def _prepare_keep(case, rng, gen):
    base, nodes, accepted = _keep_sizes(case, rng)
    bs = case["block_size"]
    lens = base + nodes
    width = -(-(case["ctx_hi"] + case["nodes_hi"]) // bs)
    num_blocks = case["seqs"] * width + 8
    tables, _ = _tables(lens, bs, width, num_blocks, rng)
    path = np.full((case["seqs"], case["accept_hi"]), -1, dtype=np.int32)
    for s, (n, a) in enumerate(zip(nodes, accepted)):
        # the first choices were the drafter's first (nothing moves), then later ones: a pass over rows that
        # were moved before moves the same rows again
        first = int(rng.integers(0, a + 1))
        if n - a < a - first:
            first = int(a)
        path[s, :first] = np.arange(first)
        path[s, first:a] = a + np.sort(rng.choice(int(n - a), size=int(a - first), replace=False))
    kc, vc = _pools(case, num_blocks, gen)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case=case, k_cache=kc, v_cache=vc, block_tables=_dev(tables), context_lens=_dev(lens),
                query_start=_dev(np.concatenate([[0], np.cumsum(nodes)])), accepted=_dev(path),
                num_accepted=_dev(accepted), new_lens=torch.empty(case["seqs"], **i32),
                status=torch.zeros(1, **i32), spare_slot=(num_blocks - 1) * bs)


# ---------------------------------------------------------------- one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_attn(s):
    import paged_kv_cache_377_b200 as pkv
    if "workspace" not in s:
        s["workspace"] = pkv.allocate_tree_workspace(s["q"].shape[2], device=s["q"].device)
    if s["case"]["fp8"]:
        return pkv.paged_attn_tree_fp8(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                       s["block_tables"], s["context_lens"], s["query_start"], s["tree_mask"],
                                       s["max_query_len"], s["scale"], s["workspace"])
    return pkv.paged_attn_tree(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                               s["query_start"], s["tree_mask"], s["max_query_len"], s["scale"], s["workspace"])


def _own_mask(s):
    import paged_kv_cache_377_b200 as pkv
    pkv.paged_tree_mask(s["tree_mask"], s["depths"], s["parents"], s["query_start"], s["max_query_len"], s["status"])
    return s["tree_mask"], s["depths"]


def _own_grow(s):
    import paged_kv_cache_377_b200 as pkv
    pkv.kv_tables_grow(s["block_tables"], s["context_lens"], s["new_tokens"], s["free_blocks"], s["num_free"],
                       s["new_lens"], s["query_start"], s["slot_mapping"], s["num_free_out"],
                       s["case"]["block_size"], s["status"])
    return s["block_tables"], s["new_lens"], s["query_start"], s["slot_mapping"], s["num_free_out"]


def _own_trim(s):
    import paged_kv_cache_377_b200 as pkv
    pkv.kv_tables_trim(s["block_tables"], s["context_lens"], s["keep_lens"], s["free_blocks"], s["num_free"],
                       s["num_free_out"], s["case"]["block_size"], s["status"])
    return s["free_blocks"], s["num_free_out"]


def _own_keep(s):
    import paged_kv_cache_377_b200 as pkv
    pkv.kv_cache_keep(s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"], s["query_start"],
                      s["accepted"], s["num_accepted"], s["new_lens"], s["status"])
    return _values(s["k_cache"]), _values(s["v_cache"]), s["new_lens"]


def _values(pool):
    """The pool as the values it stands for (e4m3 codes are a view of the same bytes)."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _rows_of(s):
    """(sequence, node) of each packed token."""
    qs = s["query_start"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(qs[1:].contiguous(), t, right=True)
    return seq, t - qs[seq]


def _gathered(pool, tables, scale):
    """fp32 [seqs, kv heads, table positions, head dim] of a pool."""
    x = _values(pool[tables.clamp(min=0).long()].flatten(1, 2)).float()
    if scale is not None:
        x = x * scale[:, None]
    return x.transpose(1, 2).contiguous()


def _plain_attn(s):
    c = s["case"]
    hq, hkv, d, n = c["q_heads"], c["kv_heads"], c["head_dim"], s["max_query_len"]
    k = _gathered(s["k_cache"], s["block_tables"], s.get("k_scale"))
    v = _gathered(s["v_cache"], s["block_tables"], s.get("v_scale"))
    seq, node = _rows_of(s)
    S, L = k.shape[0], k.shape[2]
    lens = s["context_lens"].long()
    qs = s["query_start"].long()
    base = lens - (qs[1:] - qs[:-1])
    # which positions each (sequence, node) sees: all committed ones, and the nodes of its mask
    at = (qs[:-1, None] + torch.arange(n, device=DEV)).clamp(max=s["q"].shape[0] - 1)
    bits = (s["tree_mask"][at][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    bits = bits.flatten(2).bool()
    t = torch.arange(L, device=DEV)
    j = (t - base[:, None]).clamp(0, bits.shape[2] - 1)
    sees = (t < base[:, None])[:, None, :] | (torch.gather(bits, 2, j[:, None, :].expand(S, n, L)) &
                                              (t < lens[:, None])[:, None, :])
    q = s["q"][at].float().view(S, n, hkv, hq // hkv, d).transpose(1, 2).reshape(S, hkv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(S, hkv, n, hq // hkv, L) * s["scale"]
    x = x.masked_fill(~sees[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    o = torch.matmul(p.flatten(2, 3), v).view(S, hkv, n, hq // hkv, d)
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-37)
    return o.transpose(1, 2).reshape(S, n, hq, d)[seq, node].to(torch.bfloat16)


def _plain_mask(s):
    qs = s["query_start"].long()
    S, n, words = qs.shape[0] - 1, s["max_query_len"], s["tree_mask"].shape[1]
    total = s["parents"].shape[0]
    t = torch.arange(total, device=DEV)
    seq = torch.searchsorted(qs[1:].contiguous(), t, right=True)
    node = t - qs[seq]
    # one step up the tree, and then twice as many with each squaring
    up = torch.zeros(S, n, n + 1, device=DEV)
    up[seq, node, s["parents"].long().remainder(n + 1)] = 1.0
    reach = up[:, :, :n] + torch.eye(n, device=DEV)
    far = 1
    while far < n:
        reach = (torch.matmul(reach, reach) > 0).float()
        far *= 2
    sees = reach[seq, node]
    bits = torch.nn.functional.pad(sees, (0, words * 32 - n)).view(total, words, 32).long()
    packed = (bits << torch.arange(32, device=DEV)).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
    return packed, (sees.sum(-1) - 1).int()


def _plain_grow(s):
    bs = s["case"]["block_size"]
    lens, new = s["context_lens"].long(), s["new_tokens"].long()
    have, want = (lens + bs - 1) // bs, (lens + new + bs - 1) // bs
    need = want - have
    taken = torch.cumsum(need, 0) - need
    cols = torch.arange(s["block_tables"].shape[1], device=DEV)
    k = taken[:, None] + cols - have[:, None]
    fresh = (cols >= have[:, None]) & (cols < want[:, None])
    popped = s["free_blocks"][(s["num_free"].long() - 1 - k).clamp(min=0)]
    tables = torch.where(fresh, popped, s["block_tables"])
    qs = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    t = torch.arange(s["slot_mapping"].shape[0], device=DEV)
    seq = torch.searchsorted(qs[1:].contiguous(), t, right=True).clamp(max=len(lens) - 1)
    pos = lens[seq] + t - qs[seq]
    block = tables[seq, (pos // bs).clamp(max=tables.shape[1] - 1)].long()
    slots = torch.where(t < qs[-1], block * bs + pos % bs, -1)
    return tables, (lens + new).int(), qs.int(), slots, (s["num_free"] - need.sum()).int()


def _plain_trim(s):
    bs = s["case"]["block_size"]
    lens, keep = s["context_lens"].long(), s["keep_lens"].long()
    have, kept = (lens + bs - 1) // bs, (keep + bs - 1) // bs
    freed = have - kept
    total = freed.sum()
    before = torch.cumsum(freed, 0) - freed
    cols = torch.arange(s["block_tables"].shape[1], device=DEV)
    k = before[:, None] + cols - kept[:, None]
    gone = (cols >= kept[:, None]) & (cols < have[:, None])
    # the first freed block ends on top: what was taken last goes back first
    stack = torch.cat([s["free_blocks"], s["free_blocks"].new_zeros(1)])
    at = torch.where(gone, s["num_free"].long() + total - 1 - k, stack.shape[0] - 1)
    stack[at] = s["block_tables"]
    return stack[:-1], (s["num_free"] + total).int()


def _plain_keep(s):
    bs = s["case"]["block_size"]
    qs = s["query_start"].long()
    nodes = qs[1:] - qs[:-1]
    base = s["context_lens"].long() - nodes
    k = torch.arange(s["accepted"].shape[1], device=DEV)
    live = k < s["num_accepted"][:, None]

    def slot(pos):
        block = torch.gather(s["block_tables"].long(), 1, pos // bs)
        return torch.where(live, block * bs + pos % bs, s["spare_slot"]).flatten()

    src = slot(torch.where(live, base[:, None] + s["accepted"], 0))
    dst = slot(torch.where(live, base[:, None] + k, 0))
    for pool in (s["k_cache"], s["v_cache"]):
        rows = pool.flatten(0, 1)
        rows[dst] = rows[src]
    return _values(s["k_cache"]), _values(s["v_cache"]), (base + s["num_accepted"]).int()


_PREPARE = dict(attn=_prepare_attn, mask=_prepare_mask, grow=_prepare_grow, trim=_prepare_trim, keep=_prepare_keep)
_OWN = dict(attn=_own_attn, mask=_own_mask, grow=_own_grow, trim=_own_trim, keep=_own_keep)
_PLAIN = dict(attn=_plain_attn, mask=_plain_mask, grow=_plain_grow, trim=_plain_trim, keep=_plain_keep)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    """Bytes read and written once and multiply-adds, for lengths drawn as prepare() draws them."""
    rng = np.random.default_rng(0)
    op, S = case["op"], case["seqs"]
    if op == "attn":
        base, nodes = _attn_sizes(case, rng)
        hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        blocks = int((-(-(base + nodes) // case["block_size"])).sum())
        kv = int((base + nodes).sum()) * hkv * d * 2 * (1 if case["fp8"] else 2)
        small = int(nodes.sum()) * (4 * hq * d + 4 * -(-case["nodes_hi"] // 32)) + 4 * blocks + 8 * S
        seen = float((nodes * (base + (nodes + 1) / 2)).sum())  # at most: a chain's
        return dict(bytes=kv + small, flops=4.0 * d * hq * seen)
    if op == "mask":
        total = int(_ragged(case["nodes_lo"], case["nodes_hi"], S, rng).sum())
        return dict(bytes=total * (8 + 4 * -(-case["nodes_hi"] // 32)) + 4 * (S + 1), flops=0)
    bs = case["block_size"]
    if op == "grow":
        lens, new = _grow_sizes(case, rng)
        taken = int((-(-(lens + new) // bs) - -(-lens // bs)).sum())
        tails = int(((lens % bs > 0) & (new > 0)).sum())
        return dict(bytes=8 * taken + 4 * tails + 16 * S + 8 * (int(new.sum()) + 5 * S // 4) + 12, flops=0)
    if op == "trim":
        lens, keep = _trim_sizes(case, rng)
        return dict(bytes=8 * int((-(-lens // bs) - -(-keep // bs)).sum()) + 8 * S + 8, flops=0)
    base, nodes, accepted = _keep_sizes(case, rng)
    row = case["kv_heads"] * case["head_dim"] * (1 if case["fp8"] else 2)
    return dict(bytes=int(accepted.sum()) * (2 * 2 * row * 0.5 + 12) + 20 * S, flops=0)  # about half of them move


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_attn(s):
    c = s["case"]
    bs, hq, hkv, d = c["block_size"], c["q_heads"], c["kv_heads"], c["head_dim"]
    g = hq // hkv
    lens, qs = s["context_lens"].tolist(), s["query_start"].tolist()
    words = s["tree_mask"].cpu().numpy()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for i, L in enumerate(lens):
        n = qs[i + 1] - qs[i]
        ids = s["block_tables"][i, :-(-L // bs)].long()
        rows = []
        for pool, scale in ((s["k_cache"], s.get("k_scale")), (s["v_cache"], s.get("v_scale"))):
            x = _values(pool[ids].reshape(-1, hkv, d)[:L]).double()
            rows.append(x if scale is None else x * scale.double()[None, :, None])
        bits = np.unpackbits(words[qs[i]:qs[i + 1]].view(np.uint8), axis=1, bitorder="little")[:, :n]
        hidden = torch.zeros(n, L, dtype=torch.bool, device=DEV)
        hidden[:, L - n:] = torch.from_numpy(bits == 0).to(DEV)
        for h in range(hkv):
            q = s["q"][qs[i]:qs[i + 1], h * g:(h + 1) * g].double()
            x = torch.einsum("ngd,td->ngt", q, rows[0][:, h]) * s["scale"]
            x[hidden[:, None, :].expand_as(x)] = -math.inf
            out[qs[i]:qs[i + 1], h * g:(h + 1) * g] = torch.softmax(x, -1) @ rows[1][:, h]
    return out


def _exact_mask(s):
    qs, parents = s["query_start"].tolist(), s["parents"].tolist()
    words = s["tree_mask"].shape[1]
    rows, depths = [], []
    for a, b in zip(qs, qs[1:]):
        seen = []
        for i in range(b - a):
            p = parents[a + i]
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        depths += [bin(x).count("1") - 1 for x in seen]
        rows += [[(x >> (32 * w)) & 0xffffffff for w in range(words)] for x in seen]
    return (torch.from_numpy(np.array(rows, dtype=np.uint32).view(np.int32)),
            torch.tensor(depths, dtype=torch.int32))


def _exact_grow(s):
    bs = s["case"]["block_size"]
    tables, stack = s["block_tables"].cpu().numpy().copy(), s["free_blocks"].tolist()
    stack = stack[:int(s["num_free"])]
    slots, starts, after = [], [0], []
    for i, (L, n) in enumerate(zip(s["context_lens"].tolist(), s["new_tokens"].tolist())):
        for t in range(L, L + n):
            if t % bs == 0:
                tables[i, t // bs] = stack.pop()
            slots.append(int(tables[i, t // bs]) * bs + t % bs)
        starts.append(starts[-1] + n)
        after.append(L + n)
    slots += [-1] * (s["slot_mapping"].shape[0] - len(slots))
    return (torch.from_numpy(tables), torch.tensor(after, dtype=torch.int32), torch.tensor(starts, dtype=torch.int32),
            torch.tensor(slots, dtype=torch.int64), torch.tensor([len(stack)], dtype=torch.int32))


def _exact_trim(s):
    bs = s["case"]["block_size"]
    tables, stack = s["block_tables"].tolist(), s["free_blocks"].tolist()
    free = int(s["num_free"])
    gone = []
    for row, L, keep in zip(tables, s["context_lens"].tolist(), s["keep_lens"].tolist()):
        gone += row[-(-keep // bs):-(-L // bs)]
    for b in reversed(gone):
        stack[free] = b
        free += 1
    return torch.tensor(stack, dtype=torch.int32), torch.tensor([free], dtype=torch.int32)


def _exact_keep(s):
    bs = s["case"]["block_size"]
    tables, path = s["block_tables"].tolist(), s["accepted"].tolist()
    qs, lens, counts = s["query_start"].tolist(), s["context_lens"].tolist(), s["num_accepted"].tolist()
    src, dst, after = [], [], []
    for i, L in enumerate(lens):
        base = L - (qs[i + 1] - qs[i])
        for k in range(counts[i]):
            for at, pos in ((src, base + path[i][k]), (dst, base + k)):
                at.append(tables[i][pos // bs] * bs + pos % bs)
        after.append(base + counts[i])
    pools = []
    for pool in (s["k_cache"], s["v_cache"]):
        rows = pool.flatten(0, 1)
        moved = rows.clone()
        moved[torch.tensor(dst, dtype=torch.long, device=DEV)] = rows[torch.tensor(src, dtype=torch.long, device=DEV)]
        pools.append(_values(moved.view_as(pool)).double())
    return pools[0], pools[1], torch.tensor(after, dtype=torch.int32)


_EXACT = dict(attn=_exact_attn, mask=_exact_mask, grow=_exact_grow, trim=_exact_trim, keep=_exact_keep)
