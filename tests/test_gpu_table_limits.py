"""The largest counts that the table calls take."""
import pytest
import torch

import paged_kv_cache_377_b200 as pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_every_block_of_the_largest_pool_is_given_back():
    """2^31 - 2 blocks of one token in one call: the loop over them steps past 2^31."""
    n = 2 ** 31 - 2
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(n, **i32).view(1, n)
    stack = torch.full((n,), -1, **i32)
    top, status = torch.zeros(1, **i32), torch.zeros(1, **i32)
    pkv.kv_tables_trim(table, torch.full((1,), n, **i32), torch.zeros(1, **i32), stack, top, top, 1, status)
    torch.cuda.synchronize()
    assert pkv.read_status(status) == 0 and int(top) == n
    chunk = 1 << 28
    for at in range(0, n, chunk):                    # the first block freed on top
        end = min(at + chunk, n)
        assert torch.equal(stack[at:end], table[0, n - end:n - at].flip(0)), at
