"""The split of a drafted-tree step between CTAs and the order of what a CTA's softmax warps tell one another,
modelled on the host (tree_split.py)."""
import random

import pytest

from tree_split import Piece, order_of, source_constant, split, unordered_join, unordered_marks

# A batch in which many CTAs end a segment cut in two and begin another one with a single iteration.
HAZARD = dict(lens=[571, 527, 355, 428, 331, 304, 438, 358, 431, 459, 551, 526, 348, 192],
              nodes=[35, 24, 13, 35, 22, 15, 15, 17, 12, 17, 26, 24, 21, 26], kv_heads=16, group=1, table_tokens=571)


def random_batch(rng):
    group = rng.choice([1, 2, 4, 7, 8])
    seqs = rng.randint(1, 24)
    nodes = [rng.randint(0, rng.choice([5, 40, 150])) for _ in range(seqs)]
    if not any(nodes):
        nodes[0] = 1
    top = rng.choice([100, 600, 600, 1500, 5000])
    lens = [n + rng.randint(0, top) for n in nodes]
    return dict(lens=lens, nodes=nodes, kv_heads=rng.choice([1, 2, 8, 16]), group=group,
                table_tokens=max(lens) + rng.randint(0, 100))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(25))
def test_every_iteration_of_every_segment_is_walked_once(seed, fp8):
    b = random_batch(random.Random(seed))
    seen = {}
    for mine in split(fp8=fp8, **b):
        for p in mine:
            for it in range(p.it0, p.it1):
                key = (p.seq, p.head, p.tile, it)
                assert key not in seen
                seen[key] = p.kind
    want = {(s, h, t, it) for s, (L, n) in enumerate(zip(b["lens"], b["nodes"])) for h in range(b["kv_heads"])
            for t in range(-(-n // (128 // b["group"]))) for it in range(-(-L // 64))}
    assert set(seen) == want


def hazards(mine, fp8, slots):
    return [x for pieces in mine if len(pieces) > 1 for x in unordered_join(pieces, fp8, slots)]


def test_the_kernel_keeps_enough_copies_of_the_join_word():
    """What a CTA's warps read at a piece's end is not overwritten for a later piece before: random batches, and one
    known to need more than one copy."""
    slots = source_constant("kPieceSlots")
    assert slots is not None, "one copy serves every piece"
    rng = random.Random(1)
    for b in [HAZARD] + [random_batch(rng) for _ in range(120)]:
        for fp8 in (False, True):
            assert hazards(split(fp8=fp8, **b), fp8, slots) == []


def test_one_copy_would_be_overwritten():
    """The model sees the fault that one copy is, and the known batch has it; over e4m3 pools the queries' splitting
    holds the warps together."""
    assert hazards(split(**HAZARD), False, 1)
    assert not hazards(split(fp8=True, **HAZARD), True, 1)
    two = [Piece(0, 0, 0, 3, 6, 6, "two"), Piece(1, 0, 0, 0, 1, 5, "two")]
    assert unordered_join(two, False, 1) == [(0, 1)]
    two[1].it1 = 2                                  # a second iteration waits for every warp
    assert unordered_join(two, False, 1) == []


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(5))
def test_notes_of_values_that_are_not_finite_are_ordered(seed, fp8):
    rng = random.Random(seed)
    pieces = [Piece(i, 0, 0, 0, n, n, "whole") for i, n in enumerate(rng.choices([1, 1, 2, 3], k=5))]
    assert unordered_marks(pieces, fp8, source_constant("kPieceSlots") or 2) == []


def test_the_order_model_knows_what_is_not_ordered():
    pieces = [Piece(0, 0, 0, 0, 1, 1, "whole"), Piece(1, 0, 0, 0, 1, 1, "whole")]
    o = order_of(pieces, False, False)
    assert o.before(("p_ready", 3, 0), ("o_full", 1, 0)) and not o.before(("end", 3, 0), ("mark", 1, 1))
    assert unordered_marks(pieces, False, 1)
