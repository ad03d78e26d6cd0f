"""Starts of a step's rows that a 32-bit difference mistakes for lengths: every call that takes them skips the sequence,
flags it and leaves the others as they are."""
import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from test_gpu_tree import DEV, SENTINEL, call, device_args
from tree_reference import assert_close, attention, make_step

TOP, BOTTOM = 2 ** 31 - 1, -2 ** 31
# (starts of three sequences, those that are consistent): in each some start lies 2^31 or more above the next one, so
# that their 32-bit difference is a small positive number
FALLS = [([0, TOP, BOTTOM, 8], [0, 0, 0]), ([0, 4, TOP, BOTTOM + 2], [1, 0, 0]), ([0, 5, TOP - 1, BOTTOM], [1, 0, 0]),
         ([BOTTOM, TOP, BOTTOM + 1, TOP], [0, 0, 0]), ([0, 2, 7, 2 ** 30], [1, 1, 0])]


def int32(x):
    return (x + 2 ** 31) % 2 ** 32 - 2 ** 31


def test_differences_of_these_starts_look_like_lengths():
    """In every list but the last, some sequence whose starts fall has a 32-bit difference of 0 to 7."""
    for starts, good in FALLS[:-1]:
        wrapped = [int32(b - a) for a, b in zip(starts, starts[1:])]
        assert any(0 <= w <= 7 and not g for w, g in zip(wrapped, good)), starts


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("starts,good", FALLS)
def test_tree_attention(starts, good, fp8):
    # the tree's own starts place each sequence's rows; only starts and the rows of consistent sequences are compared
    step = make_step(101, [40, 700, 3], [5, 5, 5], 4, 2, 64, 16, fp8=fp8, kind="chain")
    n = [b - a if g else 0 for a, b, g in zip(starts, starts[1:], good)]
    step.context_lens = torch.tensor([45, 705, 8], dtype=torch.int32)
    step.sees = [np.tril(np.ones((k, k), dtype=bool)) for k in n]
    rows = sum(n) + 4
    step.q = torch.randn(rows, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    mask = [[(1 << (i + 1)) - 1] for k in n for i in range(k)] + [[0]] * 4
    step.tree_mask = torch.tensor(mask, dtype=torch.int32)
    step.max_query_len = 7
    step.query_start = torch.tensor(starts, dtype=torch.int32)
    out = torch.full(step.q.shape, SENTINEL, dtype=torch.bfloat16, device=DEV)
    ws = pkv.allocate_tree_workspace(64, device=DEV)
    call(step, out, device_args(step), ws)
    torch.cuda.synchronize()
    assert pkv.read_status(ws) == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    ref, spread = attention(step, skip=[s for s in range(3) if not good[s]])
    got = out.double().cpu().numpy()
    live = sum(n)
    assert_close(got[:live], ref[:live], spread[:live], fp8, "the consistent sequences")
    assert (got[live:] == SENTINEL).all()


@pytest.mark.gpu
@pytest.mark.parametrize("starts,good", FALLS)
def test_masks(starts, good):
    live = sum(b - a for a, b, g in zip(starts, starts[1:], good) if g)
    mask = torch.full((live + 4, 1), -7, dtype=torch.int32, device=DEV)
    depths = torch.full((live + 4,), -7, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_tree_mask(mask, depths, torch.full((live + 4,), -1, dtype=torch.int32, device=DEV),
                        torch.tensor(starts, dtype=torch.int32, device=DEV), 7, status)
    assert pkv.read_status(status) == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    want = [1 << i for a, b, g in zip(starts, starts[1:], good) if g for i in range(b - a)]
    assert mask[:, 0].tolist() == want + [-7] * 4 and depths.tolist() == [0] * live + [-7] * 4


@pytest.mark.gpu
@pytest.mark.parametrize("starts,good", FALLS[:-1])
def test_kept_paths(starts, good):
    """(The last list is left out: these calls do not know how many rows a step has.)"""
    step = make_step(103, [20, 20, 20], [7, 7, 7], 2, 2, 64, 16)
    kc, vc = step.k_cache.to(DEV), step.v_cache.to(DEV)
    lens = torch.full((3,), -7, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    num = torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV)
    acc = torch.tensor([[0]] * 3, dtype=torch.int32, device=DEV)
    pkv.kv_cache_keep(kc, vc, step.block_tables.to(DEV), step.context_lens.to(DEV),
                      torch.tensor(starts, dtype=torch.int32, device=DEV), acc, num, lens, status)
    assert pkv.read_status(status) == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    assert lens.tolist() == [27 - (b - a) + 1 if g else 27 for a, b, g in zip(starts, starts[1:], good)]
    assert torch.equal(kc.cpu().view(torch.int16), step.k_cache.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(4, 2), (6, 2)])
@pytest.mark.parametrize("starts,good", FALLS)
def test_chunked_prefill(starts, good, heads):
    """Groups of two (tensor memory) and of three (the other kernel)."""
    n = [b - a if g else 0 for a, b, g in zip(starts, starts[1:], good)]
    step = make_step(105, [40, 700, 3], [5, 5, 5], *heads, 64, 16, kind="chain")
    step.sees = [np.tril(np.ones((k, k), dtype=bool)) for k in n]
    live = sum(n)
    step.q = torch.randn(live + 4, heads[0], 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    step.query_start = torch.tensor(starts, dtype=torch.int32)
    out = torch.full(step.q.shape, SENTINEL, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_attn_prefill(out, step.q.to(DEV), step.k_cache.to(DEV), step.v_cache.to(DEV), step.block_tables.to(DEV),
                           step.context_lens.to(DEV), step.query_start.to(DEV), 7, step.scale, status)
    torch.cuda.synchronize()
    assert pkv.read_status(status) == pkv.PKV_STATUS_BAD_CONTEXT_LEN
    ref, spread = attention(step, skip=[s for s in range(3) if not good[s]])
    got = out.double().cpu().numpy()
    assert_close(got[:live], ref[:live], spread[:live], False, "the consistent sequences")
    assert (got[live:] == SENTINEL).all()
