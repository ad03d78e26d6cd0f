"""kv_tables_grow and kv_tables_trim at the sizes where their kernels change how they work."""
import numpy as np
import pytest
import torch

import paged_kv_cache_377_b200 as pkv
from test_gpu_tables import Tables, trim

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,blocks_hi,bs", [(1000, 60, 16), (1024, 40, 2), (1500, 70, 1), (3, 24000, 1)])
def test_growth_of_over_sixteen_thousand_blocks(seqs, blocks_hi, bs):
    """More than two blocks for every thread of the cluster: a thread takes four in a row, across sequences' borders,
    sequences without a new block and a last turn that is not full."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 40, size=seqs)
    add = rng.integers(0, blocks_hi * bs + 1, size=seqs)
    if seqs > 3:
        add[rng.random(seqs) < 0.2] = 0
    else:
        add[:] = blocks_hi * bs - 1, 0, 7
    new = -(-(lens + add) // bs) - -(-lens // bs)
    while new.sum() % 4 == 0:                        # a count that four do not divide
        add[-1] += bs
        new = -(-(lens + add) // bs) - -(-lens // bs)
    assert new[:1024].sum() > 2 * 8 * 1024 and (new == 0).any()
    b = Tables(51, lens, bs, int((-(-(lens + add) // bs)).max()), int((-(-(lens + add) // bs)).sum()) + 5)
    got = b.grow(add, int(add.sum()) + 7)
    qs, slots = b.plain_grow(add)
    assert got[0] == b.lens and got[1] == qs and got[2] == slots + [-1] * 7
    b.assert_same()
    assert pkv.read_status(b.status) == 0


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("seqs,bs,ctx", [(1000, 1, 60), (1024, 16, 900), (1500, 1, 60), (1, 1, 50000)])
def test_trim_of_over_sixteen_thousand_blocks(seqs, bs, ctx, in_place):
    rng = np.random.default_rng(seqs + 1)
    lens = rng.integers(ctx // 2, ctx + 1, size=seqs)
    keep = rng.integers(0, 5, size=seqs)
    still = rng.random(seqs) < (0.2 if seqs > 1 else 0)
    keep[still] = lens[still]
    gone = -(-lens // bs) - -(-keep // bs)
    while gone.sum() % 4 == 0:
        keep[int(np.argmax(gone))] += bs
        gone = -(-lens // bs) - -(-keep // bs)
    assert gone[:1024].sum() > 2 * 8 * 1024
    b = Tables(53, lens, bs, -(-ctx // bs), int((-(-lens // bs)).sum()) + 9)
    b.plain_trim(keep)
    left = trim(b, keep, in_place)
    b.num_free.fill_(left)
    b.assert_same()
    assert pkv.read_status(b.status) == 0


@pytest.mark.parametrize("seqs", [8192, 8193, 20000])
def test_slots_of_more_sequences_than_starts_fit_shared_memory(seqs):
    rng = np.random.default_rng(seqs)
    lens, add = rng.integers(0, 30, size=seqs), rng.integers(0, 6, size=seqs)
    b = Tables(55, lens, 16, 3, int((-(-(lens + add) // 16)).sum()) + 1)
    slots = max(int(add.sum()), 16384) + 11
    got = b.grow(add, slots)
    qs, want = b.plain_grow(add)
    assert got[0] == b.lens and got[1] == qs and got[2] == want + [-1] * (slots - len(want))
    b.assert_same()
    assert pkv.read_status(b.status) == 0


def test_bad_ids_of_a_step_of_many_sequences_are_flagged():
    b = Tables(57, np.full(9000, 3), 16, 2, 9000 + 40)
    b.block_tables[8999, 0] = 10 ** 6
    got = b.grow(np.full(9000, 2), 18000)
    assert pkv.read_status(b.status) == pkv.PKV_STATUS_BAD_BLOCK_ID
    assert [i for i, s in enumerate(got[2]) if s < 0] == [17998, 17999]


@pytest.mark.parametrize("slots", [16384, 16385])
def test_either_side_of_where_the_second_kernel_takes_over(slots):
    rng = np.random.default_rng(slots)
    lens, add = rng.integers(0, 100, size=300), np.full(300, 54)
    b = Tables(59, lens, 16, 10, 300 * 10)
    got = b.grow(add, slots)
    qs, want = b.plain_grow(add)
    assert got[0] == b.lens and got[1] == qs and got[2] == want + [-1] * (slots - len(want))
    b.assert_same()
