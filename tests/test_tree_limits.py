"""The largest sizes that the drafted-tree calls take: one step further is refused before any CUDA call."""
import pytest

from test_tree_abi import _tree, err


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
