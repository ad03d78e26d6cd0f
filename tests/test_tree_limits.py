"""The largest sizes that the drafted-tree calls take: one step further is refused before any CUDA call."""
import ctypes

import pytest

from paged_kv_cache_377_b200 import tree
from test_tree_abi import P, _tree, err


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [16, 32])
def test_tables_whose_last_iteration_passes_32_bits(bs, fp8):
    """Contexts are walked 64 positions at a time: a length within 63 of 2^31 has no end of its last iteration."""
    most = (2 ** 31 - 64) // bs
    last = 2 ** 31 // bs - 1
    assert (most * bs + 63) // 64 * 64 < 2 ** 31 <= ((most + 1) * bs + 63) // 64 * 64
    for mb in sorted({most + 1, last}):
        assert mb * bs <= 2 ** 31 - 1
        assert _tree(fp8, MB=mb, bs=bs) == -1 and "2^31 - 64" in err(), err()


def test_a_pool_of_as_many_blocks_as_sums_saturate_at():
    args = [P] * 6 + [4, 8, 1, 2 ** 31 - 1, P, None]
    assert tree._lib().kv_tables_trim(*args) == -1 and "2^31 - 1" in err(), err()


def test_steps_over_the_blocks_of_the_largest_pool_end():
    """The trim kernel's loop in its own 32-bit arithmetic: 8 CTAs of 1024 threads, four blocks a thread. Signed, the
    step behind the last block of the largest pool is negative, and the loop goes on."""
    blocks, step = 2 ** 31 - 2, 8 * 1024 * 4
    last = (blocks - 1) // step * step               # thread 0's last turn
    assert not (last + step) % 2 ** 32 < blocks
    assert (last + step + 2 ** 31) % 2 ** 32 - 2 ** 31 < blocks


@pytest.mark.parametrize("at,words", [(3, 4), (4, 5), (5, 32), (6, 4), (2, 32)])
@pytest.mark.parametrize("end", ["first", "last"])
def test_new_lengths_in_an_inputs_memory_are_refused(at, words, end):
    """context_lens, query_start, accepted, num_accepted, block_tables: a CTA writes a length that others of its
    sequence have not read the inputs of yet. One word in common is enough."""
    args = [P, P, *(ctypes.c_void_p(1 << (20 + i)) for i in range(6)), 4, 8, 2, 64, 2, 16, 8, 64, P, None]
    start = args[at].value
    args[7] = ctypes.c_void_p(start - 12 if end == "first" else start + 4 * (words - 1))
    assert tree._lib().kv_cache_keep(*args) == -1 and "new_lens" in err(), err()
