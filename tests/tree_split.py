"""The tree kernel's split of a step between its CTAs, and what orders a CTA's softmax warps, on the host."""
from __future__ import annotations

import dataclasses
import os
import re

import paged_kv_cache_377_b200 as pkv

SMS = 148
TOKENS = 64      # positions of one iteration
WARPS = 4        # softmax warps


def source_constant(name):
    """A whole-number constant of the kernel's source; None where it has no such constant."""
    path = os.path.join(os.path.dirname(pkv.__file__), "csrc", "tree.cu")
    with open(path) as f:
        m = re.search(rf"constexpr int {name} = (\d+);", f.read())
    return int(m.group(1)) if m else None


@dataclasses.dataclass
class Piece:
    seq: int
    head: int
    tile: int
    it0: int
    it1: int
    nit: int
    kind: str        # "whole", "two" (one of a segment's two pieces) or "many" (one of three or more)


def split(lens, nodes, kv_heads, group, table_tokens, fp8=False, max_query_len=None):
    """Per CTA the pieces that it works on, in order (one launch; all sequences consistent)."""
    tile_drafts = 128 // group
    mq = max(nodes) if max_query_len is None else max_query_len
    lists = 2 if mq > tile_drafts else 1
    cost = 7 if fp8 else 4
    most_it = -(-table_tokens // TOKENS)
    whole = most_it <= 8
    min_weight = 1 if whole else 4
    tiles_of = [-(-n // tile_drafts) for n in nodes]
    most_tiles = -(-mq // tile_drafts)
    per_seq = kv_heads * most_tiles * (most_it + cost)
    bound = len(lens) * kv_heads * most_tiles if whole else len(lens) * per_seq // min_weight + 1
    grid = min(2 * SMS, 320, bound)
    if lists == 2:
        grid = max(grid, 3)
    # the segments of a list, in order: the pairs' tiles (walked twice), then what has no partner
    paired, alone = [], []
    for s, t in enumerate(tiles_of):
        for h in range(kv_heads):
            paired += [(s, h, 2 * i) for i in range(t // 2 if lists == 2 else 0)]
        if (t if lists == 1 else t % 2) and t:
            alone += [(s, h, t - 1) for h in range(kv_heads)]
    nit = [-(-L // TOKENS) for L in lens]
    wp, wa = (sum(nit[s] + cost for s, _, _ in x) for x in (paired, alone))
    W = 2 * wp + wa
    C = max((2 if wp else 0) + (1 if wa else 0), min(grid, -(-W // min_weight)))
    k = 0
    if wp:
        k = C // 2 if not wa else min(max((2 * C * wp + W) // (2 * W), 1), (C - 1) // 2)
    out = []
    for segments, second, total, ctas in ((paired, 0, wp, k), (paired, 1, wp, k), (alone, 0, wa, C - 2 * k)):
        if not total:
            continue
        bounds = [total * i // ctas for i in range(ctas + 1)]
        for c in range(ctas):
            x0, x1, at, mine = bounds[c], bounds[c + 1], 0, []
            for s, h, t in segments:
                w = nit[s] + cost
                lo, hi = max(x0, at), min(x1, at + w)
                if whole:
                    lo, hi = (at, at + w) if x0 <= at < x1 else (0, 0)
                if lo < hi:
                    it0, it1 = max(0, lo - at - cost), max(0, hi - at - cost)
                    if it1 > it0:
                        kind = "whole"
                        if it1 - it0 < nit[s]:
                            first, end = at + cost, at + w          # where the iterations begin and end
                            owners = sum(1 for i in range(ctas) if bounds[i] < end and bounds[i + 1] > first)
                            kind = "two" if owners == 2 else "many"
                        mine.append(Piece(s, h, t + second, it0, it1, nit[s], kind))
                at += w
            out.append(mine)
    return out


class Order:
    """What happens before what in a CTA: program order of the softmax warps and of the warp that issues the MMAs,
    and an edge from every arrival to the waits that need it."""

    def __init__(self):
        self.after = {}

    def edge(self, a, b):
        self.after.setdefault(a, []).append(b)

    def chain(self, events):
        for a, b in zip(events, events[1:]):
            self.edge(a, b)

    def before(self, a, b):
        seen, todo = {a}, [a]
        while todo:
            for n in self.after.get(todo.pop(), ()):
                if n == b:
                    return True
                if n not in seen:
                    seen.add(n)
                    todo.append(n)
        return False


def order_of(pieces, fp8, noted):
    """The order of a CTA with these pieces. Events: ("write", p) and ("read", w, p) of the word that says which piece
    of a segment cut in two comes first, ("mark", w, p) and ("look", w, p) of the note that a value is not finite
    (at the earliest and the latest place), and ("wipe", p). The warps only meet before the wipe, and wipe, where a
    value was ``noted``."""
    o = Order()
    first, total = [], 0
    for p in pieces:
        first.append(total)
        total += p.it1 - p.it0
    piece_of = [i for i, p in enumerate(pieces) for _ in range(p.it1 - p.it0)]
    starts = set(first)
    # the MMA warp: S one ahead of P V; over e4m3 pools a piece's first S behind the last P V of the one before
    mma = [("S", 0)]
    s = 1
    for v in range(total):
        late = fp8 and s < total and s in starts
        if s < total and not late:
            mma.append(("S", s))
            s += 1
        mma.append(("V", v))
        if late:
            mma.append(("S", s))
            s += 1
    o.chain(mma)
    for w in range(WARPS):
        events = []
        for i, p in enumerate(pieces):
            if fp8:
                events.append(("q_ready", w, i))
                o.edge(("q_ready", w, i), ("S", first[i]))
            for g in range(first[i], first[i] + p.it1 - p.it0):
                events += [("s_full", w, g), ("s_free", w, g)]
                o.edge(("S", g), ("s_full", w, g))
                if g + 1 < total:
                    o.edge(("s_free", w, g), ("S", g + 1))
                if g == first[i]:
                    events.append(("mark", w, i))
                events.append(("p_ready", w, g))
                o.edge(("p_ready", w, g), ("V", g))
            if p.kind == "two":
                if w == 0:
                    events.append(("write", i))
                events += [("meet", w, i), ("met", w, i), ("read", w, i)]
                for u in range(WARPS):
                    o.edge(("meet", w, i), ("met", u, i))
            events.append(("o_full", w, i))
            o.edge(("V", first[i] + p.it1 - p.it0 - 1), ("o_full", w, i))
            events.append(("look", w, i))
            if noted:
                events += [("meet2", w, i), ("met2", w, i)]
                for u in range(WARPS):
                    o.edge(("meet2", w, i), ("met2", u, i))
                if w == 0:
                    events.append(("wipe", i))
            events.append(("end", w, i))
        o.chain(events)
    return o


def unordered_join(pieces, fp8, slots):
    """Pairs of pieces (p, q) whose join words share one of ``slots`` places, where some warp's read of p's is not
    before the write of q's."""
    two = [i for i, p in enumerate(pieces) if p.kind == "two"]
    pairs = [(p, q) for p in two for q in two if p < q and p % slots == q % slots]
    if not pairs:
        return []
    o = order_of(pieces, fp8, False)
    return [(p, q) for p, q in pairs if not all(o.before(("read", w, p), ("write", q)) for w in range(WARPS))]


def unordered_marks(pieces, fp8, slots):
    """The same of the note that a value is not finite: marks of p reach p's looks; looks and the wipe of p are
    before the marks of a later piece with the same place."""
    n, warps, bad = len(pieces), range(WARPS), []
    for noted in (False, True):
        o = order_of(pieces, fp8, noted)
        bad += [(p, p) for p in range(n) for w in warps for u in warps if not o.before(("mark", w, p), ("look", u, p))]
        for p in range(n):
            for q in range(p + slots, n, slots):
                last = [("look", w, p) for w in warps] + ([("wipe", p)] if noted else [])
                bad += [(p, q) for u in warps for e in last if not o.before(e, ("mark", u, q))]
    return bad
