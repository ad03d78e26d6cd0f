"""paged_attn_tree over rows that real heads have and random ones do not: one large weight beside thousands of small
ones, and queries that are not finite."""
import numpy as np
import pytest
import torch

from test_gpu_tree import check, run
from tree_reference import assert_close, attention, make_step
from tree_strict import excess, moments

pytestmark = pytest.mark.gpu


def sink_step(fp8, gap, at, L=8192, seqs=20, heads=16):
    """``seqs`` sequences of one draft each over the same L tokens: so many that a CTA walks about a whole context.
    Token ``at`` has a logit ``gap`` above the middle of the others', whose logits are N(0, 0.75) or so, and V = 0;
    the others' V are positive."""
    step = make_step(95, [L - 1], [1], heads, heads, 64, 16, fp8=fp8)
    p, off = int(step.block_tables[0, at // 16]), at % 16
    if fp8:
        step.k_scale[:] = 2.0 ** -4
        step.v_scale[:] = 2.0 ** -4
        step.v_cache &= 0x7F
        step.k_cache[..., 0] = 0
        step.k_cache[p, off] = 0
        step.k_cache[p, off, :, 0] = 0x78            # 256, which the scale makes 16
        step.v_cache[p, off] = 0
    else:
        step.v_cache = step.v_cache.abs()
        step.k_cache[..., 0] = 0
        step.k_cache[p, off] = 0
        step.k_cache[p, off, :, 0] = 16
        step.v_cache[p, off] = 0
    step.q = torch.randn(seqs, heads, 64, generator=torch.Generator().manual_seed(96)).to(torch.bfloat16)
    step.q[..., 0] = gap / 2                         # times 16 times the scale of 1/8
    step.block_tables = step.block_tables.repeat(seqs, 1)
    step.context_lens = step.context_lens.repeat(seqs)
    step.query_start = torch.arange(seqs + 1, dtype=torch.int32)
    step.tree_mask = torch.ones(seqs, 1, dtype=torch.int32)
    step.sees = [np.ones((1, 1), dtype=bool)] * seqs
    return step


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("at", [0, 6000])
@pytest.mark.parametrize("gap", [11, 13, 15, 17])
def test_small_weights_beside_a_large_one_add_up(gap, at, fp8):
    """What the sums' rounding to f16 may do to a weight e^-17 of the largest, 2^-24.5 of it: kept 2^7 higher it is
    2^-17.5, a step of f16 there 2^-24, so one weight is off by up to 2^-7.5 of itself and eight thousand of unlike
    ones together by 2^-7.5 / sqrt(3 x 8192), less than a tenth of the 2^-11 that is granted."""
    check(sink_step(fp8, gap, at), f"a weight {gap} nats above the others")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_row(value, fp8):
    """Zeros where the row sees nothing, NaN where it sees something (its logits are infinite or NaN), and the other
    rows as they were."""
    step = make_step(97, [0, 50, 0], [40, 8, 3], 8, 2, 128, 16, fp8=fp8, kind="any")
    ref, spread = attention(step)
    blind = [i for i in range(40) if not step.sees[0][i].any()]
    seeing = [i for i in range(40) if step.sees[0][i].sum() > 8]
    assert len(blind) > 2 and len(seeing) > 2
    hit = np.zeros(51, dtype=bool)
    for i in (blind[0], blind[2], seeing[0], seeing[2], 43):
        step.q[i, :, 5] = value
        hit[i] = True
    out, st = run(step)
    assert st == 0
    assert (out[[blind[0], blind[2]]] == 0).all()
    assert np.isnan(out[[seeing[0], seeing[2], 43]]).all()
    assert_close(out[~hit], ref[~hit], spread[~hit], fp8, "the rows beside")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("power", [10, 18, 20, 22, 23, 24, 25])
def test_logits_far_from_zero(power, fp8):
    """Logits around 2^power (in powers of two) that grow by 2^(power - 23) from one run of 64 tokens to the next, where a
    step of fp32 grows to 4: the largest weight must not leave f16's range, however the running maximum was rounded. The
    products are exact, S = 2^21 + d / 4 with d in 0 .. 15, so that the weights are as well known as elsewhere."""
    step = make_step(99, [1200, 90, 3000], [9, 16, 5], 4, 2, 64, 16, fp8=fp8, scale=2.0 ** (power - 21) * np.log(2))
    step.q[:] = 0
    step.q[..., :8] = 2.0 ** 10
    step.q[..., 8] = 0.25
    step.k_scale[:] = 1
    for s in range(3):
        t = torch.arange(int(step.context_lens[s]))
        rows = torch.zeros(len(t), 2, 64)
        rows[..., :8] = 256
        rows[..., 8] = (t // 64 % 16)[:, None].float()
        keys = rows.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else rows.to(torch.bfloat16)
        step.k_cache[step.block_tables[s].long()[t // 16], t % 16] = keys
    out, st = run(step)
    assert st == 0
    ref, square = moments(step)
    assert excess(out, ref, square, fp8) < 1
