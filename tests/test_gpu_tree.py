"""paged_attn_tree and paged_attn_tree_fp8 against a plain fp64 form."""
import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from tree_reference import assert_close, attention, make_step

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENTINEL = 123.0


def device_args(step):
    names = ["q", "k_cache", "v_cache"] + (["k_scale", "v_scale"] if step.fp8 else []) + \
        ["block_tables", "context_lens", "query_start", "tree_mask"]
    return [getattr(step, n).to(DEV) for n in names]


def call(step, out, args, ws, stream=None):
    fn = pkv.paged_attn_tree_fp8 if step.fp8 else pkv.paged_attn_tree
    fn(out, *args, step.max_query_len, step.scale, ws, stream=stream)


def run(step):
    out = torch.full(step.q.shape, SENTINEL, dtype=torch.bfloat16, device=DEV)
    ws = pkv.allocate_tree_workspace(step.q.shape[2], device=DEV)
    call(step, out, device_args(step), ws)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), pkv.read_status(ws)


def check(step, what):
    out, st = run(step)
    assert st == 0
    ref, spread = attention(step)
    live = int(step.query_start[-1])
    assert_close(out[:live], ref[:live], spread[:live], step.fp8, what)
    assert (out[live:] == SENTINEL).all(), f"{what}: rows behind the last sequence were written"


BASE = [0, 5, 64, 130, 0, 17, 1, 500, 63]
NODES = [1, 7, 16, 33, 64, 0, 1, 65, 2]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8])
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_trees_match_the_plain_form(G, D, bs, fp8):
    check(make_step(100 * G + D + bs, BASE, NODES, 2 * G, 2, D, bs, fp8=fp8, tail_rows=3), f"G={G} D={D} bs={bs}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["chain", "any"])
@pytest.mark.parametrize("G", [4, 5])
def test_chains_and_arbitrary_masks(kind, G, fp8):
    """Among the arbitrary masks: later drafts seen, rows that see nothing, garbage in the bits past n."""
    check(make_step(7, BASE, NODES, 3 * G, 3, 128, 16, fp8=fp8, kind=kind, words=4, tail_rows=1), kind)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.2, 0.01, 1.5])
def test_scales_of_either_sign_and_size(scale, fp8):
    check(make_step(11, [300, 0, 40], [20, 9, 33], 8, 2, 128, 16, fp8=fp8, scale=scale, kind="any"), f"scale {scale}")


@pytest.mark.parametrize("fp8", [False, True])
def test_one_token_drafts_are_a_decode_step(fp8):
    check(make_step(13, [0, 4, 299, 1023, 76], [1] * 5, 32, 8, 128, 16, fp8=fp8), "n = 1")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs,base,nodes,heads", [(1, 9000, 3, (4, 1)), (2, 5000, 40, (8, 2)), (3, 2500, 100, (7, 1))])
def test_long_contexts_of_few_sequences(seqs, base, nodes, heads, fp8):
    """The context is split between many CTAs and joined."""
    check(make_step(17 + seqs, [base - 37 * s for s in range(seqs)], [nodes] * seqs, *heads, 128, 32, fp8=fp8),
          f"{seqs} x {base}")


@pytest.mark.parametrize("fp8", [False, True])
def test_trees_of_many_tiles(fp8):
    """600 and 257 drafts of eight heads a group: dozens of row tiles in pairs, odd ones out, beside one-draft trees."""
    check(make_step(43, [90, 3, 700, 0], [600, 1, 257, 16], 8, 1, 64, 16, fp8=fp8), "many tiles")


@pytest.mark.parametrize("fp8", [False, True])
def test_one_and_two_tile_trees_together(fp8):
    """Contexts that are cut, some with a pair of row tiles, some with one: three groups of CTAs."""
    check(make_step(45, [3000, 2500, 10, 1800, 0], [26, 5, 19, 18, 36], 14, 2, 128, 32, fp8=fp8), "mixed tiles")


def test_one_workspace_serves_calls_of_every_kind_in_turn():
    """Batches of other shapes, head sizes and pools follow one another through one workspace, without a wait."""
    ws = pkv.allocate_tree_workspace(128, device=DEV)
    steps = [make_step(81, [5000, 40], [16, 3], 8, 2, 128, 16), make_step(82, [3000], [40], 4, 1, 64, 32, fp8=True),
             make_step(83, [20, 9, 0], [3, 5, 1], 4, 2, 64, 16), make_step(84, [900] * 5, [20] * 5, 14, 2, 128, 16, fp8=True),
             make_step(85, [2400, 2000], [70, 12], 8, 2, 128, 32)]
    runs = [(s, torch.full(s.q.shape, SENTINEL, dtype=torch.bfloat16, device=DEV), device_args(s)) for s in steps]
    for _ in range(3):
        for s, out, args in runs:
            call(s, out, args, ws)
    torch.cuda.synchronize()
    assert pkv.read_status(ws) == 0
    for s, out, _ in runs:
        ref, spread = attention(s)
        assert_close(out.double().cpu().numpy(), ref, spread, s.fp8, "in turn")


@pytest.mark.parametrize("fp8", [False, True])
def test_skewed_batch(fp8):
    rng = np.random.default_rng(3)
    base = np.concatenate([[6000, 1500], rng.integers(0, 100, size=30)])
    check(make_step(19, base, rng.integers(0, 12, size=32), 8, 2, 64, 16, fp8=fp8), "skewed")


@pytest.mark.parametrize("fp8", [False, True])
def test_many_sequences(fp8):
    rng = np.random.default_rng(5)
    check(make_step(23, rng.integers(0, 20, size=2500), rng.integers(0, 3, size=2500), 2, 1, 64, 16, fp8=fp8),
          "2500 sequences")


@pytest.mark.parametrize("D", [64, 128])
def test_every_e4m3_code(D):
    """Zeros, subnormal codes and the largest ones, of both signs, in K and in V."""
    step = make_step(27, [256, 70], [30, 5], 8, 2, D, 16, fp8=True, scale=0.004)
    rng = np.random.default_rng(27)
    for pool in (step.k_cache, step.v_cache):
        codes = torch.from_numpy(rng.integers(0, 127, size=tuple(pool.shape)) | (rng.integers(0, 2, size=tuple(pool.shape)) << 7))
        pool[:] = torch.where(pool == 0x7F, pool, codes.to(torch.uint8))
    check(step, "all codes")


def poison(step, s, drafts, nan_k, value):
    bs = step.k_cache.shape[1]
    base = int(step.context_lens[s]) - len(step.sees[s])
    for j in drafts:
        p, off = int(step.block_tables[s, (base + j) // bs]), (base + j) % bs
        if step.fp8:
            step.k_cache[p, off], step.v_cache[p, off] = 0x7F if nan_k else 0x30, 0xFF
        else:
            step.k_cache[p, off] = float("nan") if nan_k else 1.0
            step.v_cache[p, off] = value


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("base,n", [(100, 40), (0, 6), (63, 130)])
def test_what_a_row_does_not_see_is_no_part_of_it(base, n, value, fp8):
    """NaN and infinity in drafts: rows that see them are not finite, the others are what they were."""
    step = make_step(29, [base, 50], [n, 8], 8, 2, 128, 16, fp8=fp8)
    drafts = [2, 5] if n < 100 else [2, 5, 99]
    poison(step, 0, drafts, True, value)
    out, st = run(step)
    assert st == 0
    ref, spread = attention(step)
    hit = np.zeros(len(out), dtype=bool)
    hit[:n] = step.sees[0][:, drafts].any(axis=1)
    assert hit.any() and not hit.all()
    assert np.isnan(out[hit]).all()
    assert_close(out[~hit], ref[~hit], spread[~hit], fp8, "rows beside the poisoned ones")


def test_infinite_values_that_are_seen_come_through():
    """Finite keys, infinite values: the rows that see them are infinite, of their sign."""
    step = make_step(31, [70, 9], [20, 3], 4, 2, 64, 16)
    poison(step, 0, [4], False, float("inf"))
    out, st = run(step)
    assert st == 0
    hit = np.zeros(len(out), dtype=bool)
    hit[:20] = step.sees[0][:, 4]
    assert np.isposinf(out[hit]).all() and np.isfinite(out[~hit]).all()


def test_inconsistent_sequences_are_skipped_and_flagged():
    step = make_step(37, [30, 40, 50], [5, 6, 7], 4, 2, 64, 16)
    ref, spread = attention(step)
    step.context_lens[1] = 3                       # six drafts cannot end a context of three
    out, st = run(step)
    assert st == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    rows = np.r_[0:5, 11:18]
    assert_close(out[rows], ref[rows], spread[rows], False, "the consistent sequences")
    assert (out[5:11] == SENTINEL).all()
    step.context_lens[1] = 10 ** 6                 # past its table
    assert run(step)[1] == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    step.context_lens[1] = 46
    step.max_query_len = 6                         # the last sequence brings seven
    out, st = run(step)
    assert st == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    assert_close(out[:11], ref[:11], spread[:11], False, "the shorter sequences")
    assert (out[11:] == SENTINEL).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_block_is_flagged_and_not_seen(fp8):
    step = make_step(41, [100, 20], [9, 4], 4, 2, 128, 16, fp8=fp8)
    good = int(step.block_tables[0, 2])
    step.block_tables[0, 2] = step.k_cache.shape[0] + 7
    out, st = run(step)
    assert st == pkv.PKV_STATUS_BAD_BLOCK_ID
    # what is left: the same step without that block's sixteen tokens
    step.block_tables[0, 2] = good
    cut = make_step(41, [100, 20], [9, 4], 4, 2, 128, 16, fp8=fp8)
    cut.block_tables[0, 2:-1] = step.block_tables[0, 3:].clone()
    cut.context_lens[0] -= 16
    ref, spread = attention(cut)
    assert_close(out, ref, spread, fp8, "without the bad block")


def test_captured_and_replayed_on_changed_inputs():
    """One graph; lengths, trees and values change between replays; a second graph shares the workspace."""
    steps = [make_step(50 + i, base, nodes, 8, 2, 128, 16, tail_rows=t, spare_blocks=sp)
             for i, (base, nodes, t, sp) in enumerate([([2000, 3, 60], [16, 16, 8], 0, 0), ([90, 700, 5], [4, 16, 9], 11, 0),
                                                       ([0, 0, 1], [1, 0, 16], 23, 0)])]
    width = max(s.block_tables.shape[1] for s in steps)
    nb = max(s.k_cache.shape[0] for s in steps)
    q = torch.empty(40, 8, 128, dtype=torch.bfloat16, device=DEV)
    kc = torch.empty(nb, 16, 2, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    bt = torch.zeros(3, width, dtype=torch.int32, device=DEV)
    cl, qs = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    mask = torch.zeros(40, 1, dtype=torch.int32, device=DEV)
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = pkv.allocate_tree_workspace(128, device=DEV)

    def fill(s):
        q.copy_(s.q)
        kc[:s.k_cache.shape[0]].copy_(s.k_cache)
        vc[:s.k_cache.shape[0]].copy_(s.v_cache)
        bt[:, :s.block_tables.shape[1]].copy_(s.block_tables)
        cl.copy_(s.context_lens)
        qs.copy_(s.query_start)
        mask.copy_(s.tree_mask)

    graphs = []
    fill(steps[0])
    side = torch.cuda.Stream()
    for out in outs:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pkv.paged_attn_tree(out, q, kc, vc, bt, cl, qs, mask, 16, steps[0].scale, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attn_tree(out, q, kc, vc, bt, cl, qs, mask, 16, steps[0].scale, ws)
        graphs.append(g)
    for s in (steps[1], steps[0], steps[2], steps[1]):
        fill(s)
        for g, out in zip(graphs, outs):
            out.fill_(SENTINEL)
            g.replay()
        torch.cuda.synchronize()
        assert pkv.read_status(ws) == 0
        ref, spread = attention(s)
        live = int(s.query_start[-1])
        for out in outs:
            got = out.double().cpu().numpy()
            assert_close(got[:live], ref[:live], spread[:live], False, "replay")
            assert (got[live:] == SENTINEL).all()


def test_on_another_stream_and_twice_at_once():
    a = make_step(61, [3000, 10], [16, 5], 8, 2, 128, 16)
    b = make_step(67, [20, 1800], [30, 2], 8, 2, 128, 16, fp8=True)
    runs = []
    for step in (a, b):
        st = torch.cuda.Stream()
        args = device_args(step)
        out = torch.full(step.q.shape, SENTINEL, dtype=torch.bfloat16, device=DEV)
        ws = pkv.allocate_tree_workspace(128, device=DEV)
        runs.append((step, st, args, out, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for step, st, args, out, ws in runs:
            call(step, out, args, ws, stream=st)
    torch.cuda.synchronize()
    for step, _, _, out, ws in runs:
        assert pkv.read_status(ws) == 0
        ref, spread = attention(step)
        assert_close(out.double().cpu().numpy(), ref, spread, step.fp8, "two streams")


@pytest.mark.parametrize("fp8", [False, True])
def test_the_same_call_gives_the_same_bits(fp8):
    step = make_step(71, [4000, 100, 7], [16, 64, 3], 8, 2, 128, 16, fp8=fp8)
    first = run(step)[0]
    for _ in range(3):
        assert np.array_equal(run(step)[0], first)


def test_block_order_does_not_change_a_bit():
    step = make_step(73, [1500, 40], [12, 30], 8, 2, 128, 16)
    first = run(step)[0]
    perm = torch.randperm(step.k_cache.shape[0], generator=torch.Generator().manual_seed(1))
    moved = {n: torch.empty_like(getattr(step, n)) for n in ("k_cache", "v_cache")}
    for n, m in moved.items():
        m[perm] = getattr(step, n)
        setattr(step, n, m)
    live = step.block_tables >= 0
    step.block_tables[live] = perm[step.block_tables[live].long()].int()
    assert np.array_equal(run(step)[0], first)


def test_refusals():
    step = make_step(79, [20], [4], 4, 2, 64, 16)
    args = device_args(step)
    out = torch.zeros(step.q.shape, dtype=torch.bfloat16, device=DEV)
    ws = pkv.allocate_tree_workspace(64, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.paged_attn_tree(out, args[0].transpose(0, 1).contiguous().transpose(0, 1), *args[1:], 4, 1.0, ws)
    with pytest.raises(TypeError, match="k_cache"):
        pkv.paged_attn_tree(out, args[0], args[1].half(), *args[2:], 4, 1.0, ws)
    with pytest.raises(ValueError, match="tree_mask"):
        pkv.paged_attn_tree(out, *args[:-1], args[-1][:2], 4, 1.0, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attn_tree(out, *args[:-1], args[-1].cpu(), 4, 1.0, ws)
    with pytest.raises(pkv.PagedKVError, match="mask_words"):
        pkv.paged_attn_tree(out, *args, 33, 1.0, ws)
    with pytest.raises(pkv.PagedKVError, match="workspace_bytes"):
        pkv.paged_attn_tree(out, *args, 4, 1.0, ws[:128])
