"""The strict comparison itself (tree_strict.py): what the kernel's roundings make passes it, a lost run of tokens or a
mask that is not heeded does not."""
import numpy as np
import pytest

from tree_strict import excess, moments, rounded_as_the_kernel_does
from tree_strict_cases import SHAPES, edges, pieces, plant, shape_step


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("planted", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_roundings_pass(name, planted, fp8):
    step = shape_step(name, fp8)
    if planted:
        plant(step)
    ref, square = moments(step)
    assert excess(rounded_as_the_kernel_does(step), ref, square, fp8) < 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_a_lost_run_of_sixteen_tokens_does_not(name, fp8):
    step = shape_step(name, fp8)
    ref, square = moments(step)
    L = int(step.context_lens[0])
    for at in (0, (L - len(step.sees[0])) // 32 * 16):
        wrong, _ = moments(step, lost={0: list(range(at, at + 16))})
        assert excess(wrong, ref, square, fp8) > 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_a_mask_that_is_not_heeded_does_not(name, fp8):
    step = shape_step(name, fp8)
    plant(step)
    ref, square = moments(step)
    wrong, _ = moments(step, sees=[np.ones_like(a) for a in step.sees])
    assert excess(wrong, ref, square, fp8) > 10
    wrong, _ = moments(step, sees=[np.tril(np.ones_like(a)) for a in step.sees])
    assert excess(wrong, ref, square, fp8) > 10


@pytest.mark.parametrize("name", [n for n in SHAPES if n != "uncut"])
def test_one_planted_position_does_not_get_lost(name):
    """Any of the edges of the first sequence, alone."""
    step = shape_step(name, False)
    at = plant(step)[0]
    ref, square = moments(step)
    assert len(at) < 300
    for t in edges(step, 0)[::7]:
        wrong, _ = moments(step, lost={0: [t]})
        assert excess(wrong, ref, square, False) > 1.5, t


def test_the_shapes_are_cut_as_they_are_meant_to_be():
    kinds = {name: {p.kind for mine in pieces(shape_step(name, False)) for p in mine} for name in SHAPES}
    assert kinds["uncut"] == {"whole"}
    assert "many" in kinds["one long"] and "many" in kinds["two row tiles"]
    assert "two" in kinds["cut in two"]
    step = shape_step("drafts past an edge", False)
    L = int(step.context_lens[0])
    assert sum(L - len(step.sees[0]) < t < L - 1 for t in edges(step, 0)) >= 2
