"""paged_attn_tree where contexts are cut between CTAs, under a comparison that notices a single lost edge, and with
values that are not finite and bad blocks in cut contexts."""
import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from test_gpu_tree import poison, run
from tree_reference import assert_close, attention, make_step
from tree_strict import excess, moments
from tree_strict_cases import SHAPES, pieces, plant, shape_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("planted", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_every_position_counts_once(name, planted, fp8):
    step = shape_step(name, fp8)
    if planted:
        plant(step)
    out, st = run(step)
    assert st == 0
    ref, square = moments(step)
    assert excess(out, ref, square, fp8) < 1


# (committed tokens, drafts, query heads, kv heads, head dim, block size): one sequence in many pieces, in two, and with
# drafts on both sides of a cut
CUT = {"many": ([3000, 40], [40, 5], 4, 2, 128, 16), "two": SHAPES["cut in two"], "drafts": SHAPES["drafts past an edge"]}


def cut_step(name, fp8):
    base, nodes, hq, hkv, d, bs = CUT[name]
    step = make_step(121, base, nodes, hq, hkv, d, bs, fp8=fp8)
    assert ("two" if name == "two" else "many") in {p.kind for mine in pieces(step) for p in mine}
    return step


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", CUT)
def test_drafts_that_are_not_finite_in_cut_contexts(name, value, fp8):
    step = cut_step(name, fp8)
    hit = np.zeros(step.q.shape[0], dtype=bool)
    for s in range(0, len(step.sees), 2):
        n = len(step.sees[s])
        drafts = sorted({2, n // 2, n - 3})
        poison(step, s, drafts, True, value)
        hit[int(step.query_start[s]):][:n] = step.sees[s][:, drafts].any(axis=1)
    out, st = run(step)
    assert st == 0 and hit.any() and not hit.all()
    ref, spread = attention(step)
    assert np.isnan(out[hit]).all()
    assert_close(out[~hit], ref[~hit], spread[~hit], fp8, "rows beside the poisoned ones")


@pytest.mark.parametrize("name", CUT)
def test_infinite_values_come_through_joins(name):
    """Finite keys, infinite values in the first and the last draft: rows that see one of them are infinite."""
    step = cut_step(name, False)
    hit = np.zeros(step.q.shape[0], dtype=bool)
    for s in range(len(step.sees)):
        n = len(step.sees[s])
        poison(step, s, [0, n - 1], False, float("inf"))
        hit[int(step.query_start[s]):][:n] = step.sees[s][:, [0, n - 1]].any(axis=1)
    out, st = run(step)
    assert st == 0 and hit.any() and not hit.all()
    assert np.isposinf(out[hit]).all() and np.isfinite(out[~hit]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("name", CUT)
def test_bad_blocks_in_cut_contexts(name, bad, fp8):
    """The first block, one amid, those of a whole iteration, and one that holds drafts are not seen by anyone."""
    step = cut_step(name, fp8)
    bs, s = step.k_cache.shape[1], 0
    L = int(step.context_lens[s])
    nb = -(-L // bs)
    gone = sorted({0, nb // 2, *(range(4 * (nb // 8), 4 * (nb // 8) + 64 // bs)), nb - 1})
    lost = [t for b in gone for t in range(b * bs, min((b + 1) * bs, L))]
    ref, square = moments(step, lost={s: lost})
    step.block_tables[s, gone] = bad
    out, st = run(step)
    assert st == pkv.PKV_STATUS_BAD_BLOCK_ID
    assert excess(out, ref, square, fp8) < 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,nodes_hi", [(1, 3), (8, 40)])
def test_more_sequences_than_one_launch_takes_with_cut_contexts(hq, nodes_hi, fp8):
    """Two launches (over e4m3 pools three), each with contexts that are cut and joined, one behind the other."""
    rng = np.random.default_rng(131)
    base, nodes = rng.integers(0, 20, size=1100), rng.integers(0, 3, size=1100)
    base[[0, 511, 512, 700, 1023, 1024, 1099]] = [2500, 1900, 2100, 1300, 900, 2222, 1777]
    nodes[[0, 511, 512, 700, 1023, 1024, 1099]] = [nodes_hi, 1, nodes_hi, 2, nodes_hi, 3, nodes_hi]
    step = make_step(133, base, nodes, hq, 1, 64, 16, fp8=fp8, tail_rows=2)
    out, st = run(step)
    assert st == 0
    ref, square = moments(step)
    live = int(step.query_start[-1])
    assert excess(out[:live], ref[:live], square[:live], fp8) < 1
    assert (out[live:] == out[-1, 0, 0]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_as_many_drafts_as_a_sequence_may_bring(fp8):
    """4096 drafts of one sequence, beside one of the others."""
    step = make_step(135, [5, 700], [4096, 3], 2, 1, 64, 32, fp8=fp8)
    out, st = run(step)
    assert st == 0
    ref, square = moments(step)
    assert excess(out, ref, square, fp8) < 1
