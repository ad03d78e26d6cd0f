"""paged_attn_tree where segments are cut between CTAs in particular ways (tree_split.py says how)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from test_gpu_tree import DEV, SENTINEL, call, device_args
from test_tree_split import HAZARD
from tree_reference import assert_close, attention, make_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_one_iteration_pieces_behind_joined_ones(fp8):
    """CTAs that join a segment cut in two and, one iteration later, another one: many times, always the same bits."""
    n = np.asarray(HAZARD["nodes"])
    step = make_step(91, np.asarray(HAZARD["lens"]) - n, n, HAZARD["kv_heads"] * HAZARD["group"], HAZARD["kv_heads"],
                     64, 16, fp8=fp8)
    args, ws = device_args(step), pkv.allocate_tree_workspace(64, device=DEV)
    outs = [torch.full(step.q.shape, SENTINEL, dtype=torch.bfloat16, device=DEV) for _ in range(50)]
    for out in outs:
        call(step, out, args, ws)
    torch.cuda.synchronize()
    assert pkv.read_status(ws) == 0
    ref, spread = attention(step)
    assert_close(outs[0].double().cpu().numpy(), ref, spread, fp8, "joined")
    assert all(torch.equal(o, outs[0]) for o in outs)
