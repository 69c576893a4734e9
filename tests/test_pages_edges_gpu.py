"""The page calls on states that a caller should not hand over, and pools given as any
iterable."""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
from test_pages_gpu import BIT_RANGE, DEV, i32, same

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("length", [65, 100, 1000, 2 ** 31 - 1])
def test_window_release_of_a_sequence_past_its_table(length):
    """Attention cuts such a sequence to its table's 64 positions, so what a window of 30 of those attends stays."""
    tables = np.array([[0, 1, 2, 3], [4, 5, 6, -1]], np.int32)
    t, r = i32(tables), i32([1] * 7)
    pk.kv_free_window_blocks(t, r, i32([length, 40]), 4, 2, 7, 16, 30, 0)
    same(t, [[-1, -1, 2, 3], [4, 5, 6, -1]]), same(r, [0, 0, 1, 1, 1, 1, 1])
    assert pk.kv_get_device_error() == 2                       # as the attention calls flag it


def test_copy_blocks_takes_pools_from_an_iterator():
    data = torch.arange(4 * 2048, device=DEV).to(torch.uint8).view(4, 2048)
    pools = [data.clone(), data.flip(0).contiguous()]
    pk.kv_copy_blocks(iter(pools), i32([0]), i32([3]), 1, 4)
    for p in pools:
        assert torch.equal(p[3], p[0])


@pytest.mark.parametrize("size", [4096, 16, 12, 7])
def test_copy_blocks_flags_the_same_pairs_in_every_way_of_copying(size):
    """A negative source is padding, whatever its destination; a source out of range is flagged beside any."""
    rng = np.random.default_rng(size)
    data = torch.from_numpy(rng.integers(0, 256, (6, size), dtype=np.uint8)).to(DEV)
    want = data.cpu().numpy().copy()
    want[4] = want[2]
    for src, dst, bits in (([-1, -2, 2, 3], [77, 6, 4, -1], 0), ([6, 2], [1, 4], BIT_RANGE), ([2, 2], [4, 6], BIT_RANGE),
                           ([99, 2], [-1, 4], BIT_RANGE)):
        pk.kv_copy_blocks([data], i32(src), i32(dst), len(src), 6)
        same(data, want)
        assert pk.kv_get_device_error() == bits, (src, dst)
