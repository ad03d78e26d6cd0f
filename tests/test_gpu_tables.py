"""kv_tables_grow / kv_tables_trim, paged_tree_mask and kv_cache_keep against plain Python, and a run of all of them."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from tree_reference import ancestors, assert_close, attention, make_step, pack, Step

pytestmark = pytest.mark.gpu

DEV = "cuda"


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).to(DEV)


class Tables:
    """A batch's tables with a stack of free blocks, on the device, and the same in plain Python."""

    def __init__(self, seed, lens, bs, width, num_blocks):
        rng = np.random.default_rng(seed)
        perm = rng.permutation(num_blocks)
        self.bs, self.width, self.nb = bs, width, num_blocks
        self.lens = [int(x) for x in lens]
        self.rows, at = [], 0
        for L in self.lens:
            k = -(-L // bs)
            self.rows.append([int(x) for x in perm[at:at + k]])
            at += k
        self.stack = [int(x) for x in perm[at:]]
        t = np.full((len(lens), width), -1)
        for s, r in enumerate(self.rows):
            t[s, :len(r)] = r
        self.block_tables, self.context_lens = dev(t), dev(np.asarray(lens))
        f = np.full(num_blocks, -1)
        f[:len(self.stack)] = self.stack
        self.free_blocks, self.num_free = dev(f), dev([len(self.stack)])
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def grow(self, new, num_slots, in_place=True):
        S = len(self.lens)
        qs = torch.full((S + 1,), -7, dtype=torch.int32, device=DEV)
        slots = torch.full((num_slots,), -7, dtype=torch.int64, device=DEV)
        lens = self.context_lens if in_place else torch.full_like(self.context_lens, -7)
        left = self.num_free if in_place else torch.full_like(self.num_free, -7)
        pkv.kv_tables_grow(self.block_tables, self.context_lens, dev(new), self.free_blocks, self.num_free, lens, qs,
                           slots, left, self.bs, self.status)
        torch.cuda.synchronize()
        return lens.tolist(), qs.tolist(), slots.tolist(), int(left)

    def plain_grow(self, new):
        slots, qs = [], [0]
        for s, n in enumerate(new):
            for t in range(self.lens[s], self.lens[s] + n):
                if t % self.bs == 0:
                    self.rows[s].append(self.stack.pop())
                slots.append(self.rows[s][t // self.bs] * self.bs + t % self.bs)
            self.lens[s] += int(n)
            qs.append(qs[-1] + int(n))
        return qs, slots

    def plain_trim(self, keep):
        gone = []
        for s, k in enumerate(keep):
            gone += self.rows[s][-(-k // self.bs):]
            self.rows[s] = self.rows[s][:-(-k // self.bs)]
            self.lens[s] = int(k)
        self.stack += gone[::-1]

    def assert_same(self):
        t = self.block_tables.tolist()
        for s, r in enumerate(self.rows):
            assert t[s][:len(r)] == r, s
        assert int(self.num_free) == len(self.stack)
        assert self.free_blocks.tolist()[:len(self.stack)] == self.stack


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("seqs,bs,ctx,new,extra", [
    (1, 16, 0, 1, 0), (4, 16, 33, 7, 3), (256, 16, 300, 1, 0), (1000, 32, 90, 60, 17), (1024, 16, 40, 3, 1),
    (1025, 1, 9, 4, 100), (2300, 7, 20, 30, 5000), (3, 16, 100, 20000, 11), (5, 16, 50, 0, 8)])
def test_grow_matches_plain_python(seqs, bs, ctx, new, extra, in_place):
    rng = np.random.default_rng(seqs + bs)
    lens, add = rng.integers(0, ctx + 1, size=seqs), rng.integers(0, new + 1, size=seqs)
    width = -(-(ctx + new) // bs) + 1
    b = Tables(1, lens, bs, width, int((-(-(lens + add) // bs)).sum()) + 2)
    before = b.context_lens.tolist(), int(b.num_free)
    got = b.grow(add, int(add.sum()) + extra, in_place)
    if not in_place:
        assert (b.context_lens.tolist(), int(b.num_free)) == before
        b.num_free.fill_(got[3])
    qs, slots = b.plain_grow(add)
    assert got[0] == b.lens and got[1] == qs and got[2] == slots + [-1] * extra
    b.assert_same()
    assert pkv.read_status(b.status) == 0


def test_grow_of_no_sequences_is_an_empty_step():
    b = Tables(2, [], 16, 4, 5)
    assert b.grow(np.zeros(0, dtype=np.int64), 3) == ([], [0], [-1] * 3, 5)


@pytest.mark.parametrize("why,bit", [("blocks", 64), ("slots", 128), ("table", 2), ("negative", 2), ("length", 2)])
def test_grow_is_all_or_nothing(why, bit):
    lens = np.array([10, 40, 0, 31] * 300)
    add = np.array([7, 0, 16, 2] * 300)
    taken = int((-(-(lens + add) // 16) - -(-lens // 16)).sum())
    b = Tables(3, lens, 16, 4, int((-(-lens // 16)).sum()) + taken - (1 if why == "blocks" else 0))
    if why == "table":
        add[1199] = 34                       # 65 tokens in a table of 64
    if why == "negative":
        add[5] = -1
    if why == "length":
        b.context_lens[700] = -3
    tables, stack = b.block_tables.clone(), b.free_blocks.clone()
    before, free = b.context_lens.tolist(), int(b.num_free)
    slots = int(np.maximum(add, 0).sum()) - (1 if why == "slots" else 0)
    got = b.grow(add, slots)
    assert pkv.read_status(b.status) & bit
    assert got == (before, [0] * 1201, [-1] * slots, free)
    assert torch.equal(tables, b.block_tables) and torch.equal(stack, b.free_blocks)


@pytest.mark.parametrize("why,bit", [("blocks", 64), ("negative", 2)])
def test_large_steps_are_all_or_nothing_too(why, bit):
    """More slots than one cluster takes: the second kernel writes nothing but -1."""
    lens, add = np.full(500, 21), np.full(500, 60)
    b = Tables(31, lens, 16, 6, 500 * 2 + (500 * 4 - 1 if why == "blocks" else 3000))
    if why == "negative":
        add[77] = -5
    tables, before, free = b.block_tables.clone(), b.context_lens.tolist(), int(b.num_free)
    assert b.grow(add, 30001) == (before, [0] * 501, [-1] * 30001, free)
    assert pkv.read_status(b.status) == bit and torch.equal(tables, b.block_tables)


def test_bad_ids_of_a_large_step_are_flagged():
    b = Tables(32, [5, 16], 16, 2000, 4100)
    b.free_blocks[int(b.num_free) - 2] = 5000      # the second block taken
    got = b.grow([20000, 30], 20040)
    assert pkv.read_status(b.status) == pkv.PKV_STATUS_BAD_BLOCK_ID
    bad = [i for i, s in enumerate(got[2][:20030]) if s < 0]
    assert bad == list(range(27, 43)) and got[2][20030:] == [-1] * 10


def test_grow_and_trim_back_to_back_without_a_wait():
    """A hundred steps that lean on one another, each started while the one before ends."""
    rng = np.random.default_rng(33)
    lens = rng.integers(0, 50, size=300)
    b = Tables(33, lens, 16, 20, 5000)
    S = 300
    qs = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(20000, dtype=torch.int64, device=DEV)
    adds = [rng.integers(0, 9, size=S) for _ in range(50)]
    keeps, L = [], lens.copy()
    for a in adds:
        L = L + a
        keeps.append(np.maximum(L - rng.integers(0, 7, size=S), 0))
        L = keeps[-1]
    dadds, dkeeps = [dev(a) for a in adds], [dev(k) for k in keeps]
    for a, k in zip(dadds, dkeeps):
        pkv.kv_tables_grow(b.block_tables, b.context_lens, a, b.free_blocks, b.num_free, b.context_lens, qs, slots,
                           b.num_free, 16, b.status)
        pkv.kv_tables_trim(b.block_tables, b.context_lens, k, b.free_blocks, b.num_free, b.num_free, 16, b.status)
        b.context_lens.copy_(k)
    torch.cuda.synchronize()
    for a, k in zip(adds, keeps):
        want = b.plain_grow(a)
        b.plain_trim(k)
    assert slots.tolist()[:len(want[1])] == want[1] and qs.tolist() == want[0]
    b.assert_same()
    assert pkv.read_status(b.status) == 0


def test_bad_ids_and_counts_are_flagged():
    b = Tables(4, [5, 16], 16, 4, 10)
    b.free_blocks[int(b.num_free) - 1] = 99
    b.block_tables[0, 0] = -4
    got = b.grow([3, 2], 5)
    assert got[2] == [-1] * 5 and pkv.read_status(b.status) == pkv.PKV_STATUS_BAD_BLOCK_ID
    b = Tables(4, [5, 16], 16, 4, 10)
    b.num_free.fill_(11)
    assert b.grow([3, 2], 5)[1] == [0, 0, 0] and pkv.read_status(b.status) == pkv.PKV_STATUS_BAD_BLOCK_ID


def trim(b, keep, in_place=True):
    left = b.num_free if in_place else torch.full_like(b.num_free, -7)
    pkv.kv_tables_trim(b.block_tables, b.context_lens, dev(keep), b.free_blocks, b.num_free, left, b.bs, b.status)
    torch.cuda.synchronize()
    return int(left)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("seqs,bs,ctx,drop", [(1, 16, 40, 40), (4, 16, 33, 7), (1000, 16, 300, 20), (1025, 32, 90, 91),
                                              (2300, 1, 9, 9), (3, 16, 60000, 60000), (6, 16, 0, 0)])
def test_trim_matches_plain_python(seqs, bs, ctx, drop, in_place):
    rng = np.random.default_rng(seqs + bs)
    lens = rng.integers(0, ctx + 1, size=seqs)
    keep = np.maximum(lens - rng.integers(0, drop + 1, size=seqs), 0)
    b = Tables(5, lens, bs, max(-(-ctx // bs), 1), int((-(-lens // bs)).sum()) + 3)
    b.plain_trim(keep)
    left = trim(b, keep, in_place)
    b.num_free.fill_(left)
    b.assert_same()
    assert pkv.read_status(b.status) == 0


def test_a_grow_undone_by_a_trim_leaves_the_stack_as_it_was():
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 200, size=1500)
    b = Tables(6, lens, 16, 20, 30000)
    stack, free = b.free_blocks.clone(), int(b.num_free)
    lens0 = b.context_lens.clone()
    add = rng.integers(0, 100, size=1500)
    b.grow(add, int(add.sum()))
    assert int(b.num_free) < free
    trim(b, lens0.cpu().numpy())
    assert int(b.num_free) == free and torch.equal(stack, b.free_blocks)


@pytest.mark.parametrize("why,bit", [("more", 2), ("negative", 2), ("twice", 1)])
def test_trim_is_all_or_nothing(why, bit):
    b = Tables(7, [40, 50, 16], 16, 4, 9)
    keep = [16, 50, 0]
    if why == "more":
        keep[1] = 51
    if why == "negative":
        keep[1] = -1
    if why == "twice":
        b.num_free.fill_(9)
    stack, free = b.free_blocks.clone(), int(b.num_free)
    assert trim(b, keep) == free and torch.equal(stack, b.free_blocks)
    assert pkv.read_status(b.status) == bit


def test_trim_of_a_bad_entry_is_flagged():
    b = Tables(8, [40], 16, 4, 5)
    b.block_tables[0, 1] = 77
    free = int(b.num_free)
    assert trim(b, [0]) == free + 3
    got = b.free_blocks.tolist()[free:free + 3]
    assert got == [b.rows[0][2], -1, b.rows[0][0]] and pkv.read_status(b.status) == pkv.PKV_STATUS_BAD_BLOCK_ID


def random_parents(rng, n, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "roots":
        return [-1] * n
    return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]


@pytest.mark.parametrize("kind", ["tree", "chain", "roots"])
@pytest.mark.parametrize("nodes,words", [([1], 1), ([7, 0, 3, 16], 1), ([32, 31, 33], 2), ([64, 5, 65, 130], 6),
                                         ([1000, 2, 4096], 128), ([3] * 700, 1)])
def test_masks_match_plain_python(nodes, words, kind):
    rng = np.random.default_rng(len(nodes) + words)
    parents = [random_parents(rng, n, kind) for n in nodes]
    total = sum(nodes)
    mask = torch.full((total + 2, words), -7, dtype=torch.int32, device=DEV)
    depths = torch.full((total + 2,), -7, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    flat = dev(sum(parents, []) + [-1, -1])
    pkv.paged_tree_mask(mask, depths, flat, dev(np.concatenate([[0], np.cumsum(nodes)])), max(nodes), status)
    assert pkv.read_status(status) == 0
    sees = [ancestors(p) for p in parents]
    want = np.concatenate([pack(a, words) for a in sees])
    assert np.array_equal(mask.cpu().numpy()[:total], want)
    assert depths.tolist()[:total] == [int(r.sum()) - 1 for a in sees for r in a]
    assert (mask[total:] == -7).all() and (depths[total:] == -7).all()


def test_bad_parents_count_as_roots_and_are_flagged():
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mask = torch.zeros(6, 1, dtype=torch.int32, device=DEV)
    depths = torch.zeros(6, dtype=torch.int32, device=DEV)
    pkv.paged_tree_mask(mask, depths, dev([-1, 1, 5, -2, 0, 4]), dev([0, 6]), 6, status)
    assert pkv.read_status(status, clear=True) == pkv.PKV_STATUS_BAD_TREE
    assert mask[:, 0].tolist() == [1, 2, 4, 8, 17, 49] and depths.tolist() == [0, 0, 0, 0, 1, 2]
    mask.fill_(-7)
    pkv.paged_tree_mask(mask, depths, dev([-1] * 6), dev([0, 4, 7]), 4, status)      # seven rows of six
    assert pkv.read_status(status, clear=True) == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    assert mask[:, 0].tolist() == [1, 2, 4, 8, -7, -7]
    pkv.paged_tree_mask(mask, depths, dev([-1] * 6), dev([0, 4, 2]), 4, status)
    assert pkv.read_status(status) == pkv.PKV_STATUS_BAD_CONTEXT_LEN


def keep_case(seed, nodes, base, bs, hkv, d, fp8, paths):
    step = make_step(seed, base, nodes, hkv, hkv, d, bs, fp8=fp8)
    width = max([len(p) for p in paths] + [1])
    acc = np.full((len(paths), width), -1)
    for s, p in enumerate(paths):
        acc[s, :len(p)] = p
    return step, dev(acc), dev([len(p) for p in paths])


def plain_keep(step, paths, pool):
    bs = pool.shape[1]
    rows = pool.clone().view(torch.uint8 if pool.dtype == torch.uint8 else torch.int16).flatten(0, 1)
    old = rows.clone()
    for s, p in enumerate(paths):
        base = int(step.context_lens[s]) - len(step.sees[s])
        at = [int(step.block_tables[s, (base + i) // bs]) * bs + (base + i) % bs for i in range(len(step.sees[s]))]
        for k, i in enumerate(p):
            rows[at[k]] = old[at[i]]
    return rows


def run_keep(step, acc, num, new_lens=True):
    kc, vc = step.k_cache.to(DEV), step.v_cache.to(DEV)
    out = torch.full((len(step.sees),), -7, dtype=torch.int32, device=DEV) if new_lens else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_cache_keep(kc, vc, step.block_tables.to(DEV), step.context_lens.to(DEV), step.query_start.to(DEV), acc, num,
                      out, status)
    torch.cuda.synchronize()
    bits = torch.uint8 if step.fp8 else torch.int16
    return kc.cpu().view(bits).flatten(0, 1), vc.cpu().view(bits).flatten(0, 1), out, pkv.read_status(status)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (8, 128, 16), (3, 64, 32), (40, 128, 32), (5, 16, 7)])
def test_kept_paths_match_plain_python(hkv, d, bs, fp8):
    """Paths that overlap their own targets, identities, empty ones, ends of blocks, and longer than 128 rows."""
    nodes = [64, 7, 1, 0, 300, 16, 12]
    base = [30, 0, 15, 20, 5, 16, 33]
    rng = np.random.default_rng(9)
    paths = [[1, 2, 4, 9, 10, 63], list(range(7)), [0], [], sorted(rng.choice(300, size=200, replace=False).tolist()),
             [], [11]]
    step, acc, num = keep_case(10, nodes, base, bs, hkv, d, fp8, paths)
    k, v, lens, st = run_keep(step, acc, num)
    assert st == 0
    assert torch.equal(k, plain_keep(step, paths, step.k_cache)) and torch.equal(v, plain_keep(step, paths, step.v_cache))
    assert lens.tolist() == [b + len(p) for b, p in zip(base, paths)]
    again = run_keep(step, acc, num, new_lens=False)
    assert torch.equal(again[0], k) and torch.equal(again[1], v)


@pytest.mark.parametrize("path,count,bit", [([3, 3], 2, 32), ([4, 2], 2, 32), ([2, 9], 2, 32), ([-1, 2], 2, 32),
                                            ([1, 2], 3, 32), ([1, 2], -1, 32), ([1, 8], 2, 1), (None, 2, 2)])
def test_bad_paths_move_nothing(path, count, bit):
    step, acc, num = keep_case(12, [9, 9], [10, 10], 16, 2, 64, False, [[1, 2], [1, 2]])
    num[0] = count
    if path is None:
        step.context_lens[0] = 8
    else:
        acc[0] = dev(path)
    if bit == 1:
        step.block_tables[0, 1] = 1000
    k, v, lens, st = run_keep(step, acc, num)
    assert st == bit
    only = [[], [1, 2]]
    assert torch.equal(k, plain_keep(step, only, step.k_cache)) and torch.equal(v, plain_keep(step, only, step.v_cache))
    assert lens.tolist() == [int(step.context_lens[0]), 12]


@pytest.mark.parametrize("fp8", [False, True])
def test_a_run_of_steps_as_a_server_makes_them(fp8):
    """Prompts admitted, then rounds of drafts: grow, mask, append, tree attention, an accepted path kept, the rest
    trimmed; the attention of each round and the cache at the end against plain forms that know the tokens only."""
    rng = np.random.default_rng(14)
    gen = torch.Generator().manual_seed(14)
    S, hq, hkv, d, bs, nb, width = 5, 8, 2, 128, 16, 120, 24
    b = Tables(14, [0] * S, bs, width, nb)
    kc = torch.zeros(nb, bs, hkv, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    h = torch.arange(hkv, dtype=torch.float32)
    ks, vs = (2.0 ** -6 * (1 + h)).to(DEV), (2.0 ** -6 * (2 + h)).to(DEV)
    ws = pkv.allocate_tree_workspace(d, device=DEV)
    kept = [[] for _ in range(S)]            # per sequence the committed (k, v) rows

    def append(rows, slots):
        k, v = (torch.stack([r[i] for r in rows]).to(DEV) for i in (0, 1))
        if fp8:
            pkv.kv_cache_append_fp8(k, v, kc, vc, slots, ks, vs, b.status)
        else:
            pkv.kv_cache_append(k, v, kc, vc, slots, b.status)

    def fresh(n):
        return [tuple(torch.randn(hkv, d, generator=gen).to(torch.bfloat16) for _ in range(2)) for _ in range(n)]

    def grow(new):
        qs = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
        slots = torch.zeros(int(sum(new)), dtype=torch.int64, device=DEV)
        pkv.kv_tables_grow(b.block_tables, b.context_lens, dev(new), b.free_blocks, b.num_free, b.context_lens, qs,
                           slots, b.num_free, bs, b.status)
        return qs, slots

    prompt = [40, 1, 100, 17, 64]
    _, slots = grow(prompt)
    rows = [fresh(n) for n in prompt]
    append(sum(rows, []), slots)
    for s in range(S):
        kept[s] += rows[s]
    for step_no in range(4):
        nodes = [int(x) for x in rng.integers(1, 20, size=S)]
        parents = [random_parents(rng, n, "tree") for n in nodes]
        qs, slots = grow(nodes)
        mask = torch.zeros(sum(nodes), 1, dtype=torch.int32, device=DEV)
        depths = torch.zeros(sum(nodes), dtype=torch.int32, device=DEV)
        pkv.paged_tree_mask(mask, depths, dev(sum(parents, [])), qs, max(nodes), b.status)
        rows = [fresh(n) for n in nodes]
        append(sum(rows, []), slots)
        q = torch.randn(sum(nodes), hq, d, generator=gen).to(torch.bfloat16)
        out = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV)
        args = [out, q.to(DEV), kc, vc] + ([ks, vs] if fp8 else []) + [b.block_tables, b.context_lens, qs, mask]
        (pkv.paged_attn_tree_fp8 if fp8 else pkv.paged_attn_tree)(*args, max(nodes), 1 / math.sqrt(d), ws)
        # the plain form, from the rows alone, in a cache of its own
        want = make_step(1, [len(x) for x in kept], nodes, hq, hkv, d, bs, fp8=fp8)
        want.q, want.sees, want.k_scale, want.v_scale = q, [ancestors(p) for p in parents], ks.cpu(), vs.cpu()
        for s in range(S):
            for t, row in enumerate(kept[s] + rows[s]):
                p, off = int(want.block_tables[s, t // bs]), t % bs
                for pool, x, sc in ((want.k_cache, row[0], want.k_scale), (want.v_cache, row[1], want.v_scale)):
                    pool[p, off] = (x.float() / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x
        ref, spread = attention(want)
        assert_close(out.double().cpu().numpy(), ref, spread, fp8, f"step {step_no}")
        # a path from a random leaf, cut somewhere
        paths = []
        for s in range(S):
            j, path = int(rng.integers(0, nodes[s])), []
            while j >= 0:
                path.append(j)
                j = parents[s][j]
            paths.append(path[::-1][:int(rng.integers(0, len(path) + 1))])
            kept[s] += [rows[s][j] for j in paths[s]]
        acc = np.full((S, 20), -1)
        for s, p in enumerate(paths):
            acc[s, :len(p)] = p
        lens = torch.empty(S, dtype=torch.int32, device=DEV)
        pkv.kv_cache_keep(kc, vc, b.block_tables, b.context_lens, qs, dev(acc), dev([len(p) for p in paths]), lens,
                          b.status)
        pkv.kv_tables_trim(b.block_tables, b.context_lens, lens, b.free_blocks, b.num_free, b.num_free, bs, b.status)
        b.context_lens.copy_(lens)
        assert lens.tolist() == [len(x) for x in kept]
        assert int(b.num_free) == nb - sum(-(-len(x) // bs) for x in kept)
    # a decode step over what is left gives what the rows give
    q = torch.randn(S, hq, d, generator=gen).to(torch.bfloat16)
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV)
    dws = pkv.allocate_workspace(S, hq, d, device=DEV)
    if fp8:
        pkv.paged_attn_decode_fp8(out, q.to(DEV), kc, vc, ks, vs, b.block_tables, b.context_lens, 1 / math.sqrt(d), dws)
    else:
        pkv.paged_attn_decode(out, q.to(DEV), kc, vc, b.block_tables, b.context_lens, 1 / math.sqrt(d), dws)
    want = make_step(2, [len(x) - 1 for x in kept], [1] * S, hq, hkv, d, bs, fp8=fp8)
    want.q, want.k_scale, want.v_scale = q, ks.cpu(), vs.cpu()
    for s in range(S):
        for t, row in enumerate(kept[s]):
            p, off = int(want.block_tables[s, t // bs]), t % bs
            for pool, x, sc in ((want.k_cache, row[0], want.k_scale), (want.v_cache, row[1], want.v_scale)):
                pool[p, off] = (x.float() / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x
    ref, spread = attention(want)
    assert_close(out.double().cpu().numpy(), ref, spread, fp8, "decode after the steps")
    # all requests end: every block is back, once
    pkv.kv_tables_trim(b.block_tables, b.context_lens, torch.zeros_like(b.context_lens), b.free_blocks, b.num_free,
                       b.num_free, bs, b.status)
    assert sorted(b.free_blocks.tolist()) == list(range(nb)) and int(b.num_free) == nb
    assert pkv.read_status(b.status) == 0 and pkv.read_status(ws) == 0


def test_a_step_is_captured_into_one_graph():
    """grow in place, append and trim captured once: replays grow the same sequences on and on."""
    lens, bs = [3, 15, 16, 0], 16
    b = Tables(15, lens, bs, 12, 48)
    qs = torch.zeros(5, dtype=torch.int32, device=DEV)
    slots = torch.zeros(12, dtype=torch.int64, device=DEV)
    new = dev([1, 5, 2, 0])
    k = torch.randn(12, 2, 64, device=DEV, dtype=torch.bfloat16)
    kc = torch.zeros(48, bs, 2, 64, device=DEV, dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)

    def step():
        pkv.kv_tables_grow(b.block_tables, b.context_lens, new, b.free_blocks, b.num_free, b.context_lens, qs, slots,
                           b.num_free, bs, b.status)
        pkv.kv_cache_append(k, k, kc, vc, slots, b.status)

    step()
    b.plain_grow([1, 5, 2, 0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for add in ([1, 5, 2, 0], [0, 1, 0, 12], [4, 4, 4, 0], [0, 0, 0, 0], [1, 1, 1, 1]):
        new.copy_(dev(add))
        g.replay()
        torch.cuda.synchronize()
        # thirteen tokens do not fit the captured step's twelve slots: that replay is an empty step
        fits = sum(add) <= 12
        assert pkv.read_status(b.status, clear=True) == (0 if fits else pkv.PKV_STATUS_OUT_OF_SLOTS)
        want_qs, want = b.plain_grow(add) if fits else ([0] * 5, [])
        assert qs.tolist() == want_qs and slots.tolist() == want + [-1] * (12 - len(want))
        assert b.context_lens.tolist() == b.lens
        b.assert_same()
        for i, sl in enumerate(want):
            assert torch.equal(kc.flatten(0, 1)[sl], k[i])


def test_refusals():
    b = Tables(16, [3, 4], 16, 4, 8)
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, qs, left = torch.zeros(2, **i32), torch.zeros(3, **i32), torch.zeros(1, **i32)
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError, match="num_seqs"):
        pkv.kv_tables_grow(b.block_tables, b.context_lens, dev([1]), b.free_blocks, b.num_free, lens, qs, slots, left,
                           16, b.status)
    with pytest.raises(TypeError, match="slot_mapping"):
        pkv.kv_tables_grow(b.block_tables, b.context_lens, dev([1, 1]), b.free_blocks, b.num_free, lens, qs, lens,
                           left, 16, b.status)
    with pytest.raises(pkv.PagedKVError, match="block_size"):
        pkv.kv_tables_grow(b.block_tables, b.context_lens, dev([1, 1]), b.free_blocks, b.num_free, lens, qs, slots,
                           left, 0, b.status)
    with pytest.raises(ValueError, match="num_seqs"):
        pkv.kv_tables_trim(b.block_tables, b.context_lens, dev([1]), b.free_blocks, b.num_free, left, 16, b.status)
    mask, depths = torch.zeros(4, 1, **i32), torch.zeros(4, **i32)
    with pytest.raises(pkv.PagedKVError, match="mask_words"):
        pkv.paged_tree_mask(mask, depths, dev([-1] * 4), dev([0, 4]), 33, b.status)
    with pytest.raises(pkv.PagedKVError, match="exceeds"):
        pkv.paged_tree_mask(mask, depths, dev([-1] * 4), dev([0, 4]), 5000, b.status)
    with pytest.raises(ValueError, match="row per token"):
        pkv.paged_tree_mask(mask, depths, dev([-1] * 3), dev([0, 4]), 4, b.status)
    pool = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(pkv.PagedKVError, match="new_lens"):
        pkv.kv_cache_keep(pool, pool.clone(), b.block_tables, b.context_lens, qs, dev([[0], [0]]), dev([1, 1]),
                          b.context_lens, b.status)
    with pytest.raises(TypeError, match="v_cache"):
        pkv.kv_cache_keep(pool, pool.byte(), b.block_tables, b.context_lens, qs, dev([[0], [0]]), dev([1, 1]), lens,
                          b.status)
