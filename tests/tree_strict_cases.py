"""Steps for the strict comparison: contexts that many CTAs share, random and with the weight planted at the edges."""
import numpy as np
import torch

from test_tree_split import HAZARD
from tree_reference import make_step
from tree_split import split

_H = np.asarray(HAZARD["nodes"])
# name -> (committed tokens, drafts, query heads, kv heads, head dim, block size)
SHAPES = {
    "one long": ([9000], [3], 4, 1, 128, 32),
    "two with a tree each": ([5000, 4963], [40, 40], 8, 2, 128, 32),
    "two row tiles": ([2500, 2463, 2426], [100, 100, 100], 7, 1, 128, 32),
    "cut in two": ((np.asarray(HAZARD["lens"]) - _H).tolist(), _H.tolist(), 16, 16, 64, 16),
    "drafts past an edge": ([3000, 520], [200, 190], 4, 2, 64, 16),
    "one and two tiles": ([3000, 2500, 10, 1800], [26, 5, 19, 18], 14, 2, 128, 32),
    "uncut": ([150, 30, 0], [20, 64, 9], 8, 2, 128, 16),
}


def shape_step(name, fp8, seed=111):
    base, nodes, hq, hkv, d, bs = SHAPES[name]
    return make_step(seed, base, nodes, hq, hkv, d, bs, fp8=fp8)


def pieces(step):
    """The step's pieces, CTA by CTA."""
    bs, hkv = step.k_cache.shape[1:3]
    n = (step.query_start[1:] - step.query_start[:-1]).tolist()
    return split(step.context_lens.tolist(), n, hkv, step.q.shape[1] // hkv, step.block_tables.shape[1] * bs, step.fp8,
                 step.max_query_len)


def edges(step, s):
    """Positions of sequence s on either side of every cut between its pieces, of the committed tokens' end, and of the
    context's two ends."""
    L = int(step.context_lens[s])
    first = L - len(step.sees[s])
    at = {0, L - 1, first - 1, first}
    for mine in pieces(step):
        for p in mine:
            if p.seq == s:
                at |= {64 * p.it0, 64 * p.it0 - 1, 64 * p.it1 - 1, 64 * p.it1}
    return sorted(t for t in at if 0 <= t < L)


def plant(step):
    """Nearly all weight, in equal parts, on the edges of each sequence and on all its drafts: one position more or less
    moves a row by V over their number. Returns the planted positions per sequence."""
    bs = step.k_cache.shape[1]
    step.q[..., 0] = 16.0
    out = []
    for s in range(len(step.sees)):
        L = int(step.context_lens[s])
        t = torch.arange(L)
        rows = step.block_tables[s].long()[t // bs], t % bs
        step.k_cache[rows[0], rows[1], :, 0] = 0
        first = L - len(step.sees[s])
        at = sorted(set(edges(step, s)) | set(range(first, L)))
        blocks, offs = rows[0][at], rows[1][at]
        step.k_cache[blocks, offs] = 0
        # 16 x 16 x scale >= 22 above logits of N(0, 1) or so (e4m3: 0x78 is 256, times scales from 2^-4 on)
        step.k_cache[blocks, offs, :, 0] = 0x78 if step.fp8 else 16.0
        out.append(at)
    return out
