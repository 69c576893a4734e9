"""Decodes over shared prefixes at the ends of what their documentation allows, against
64-bit attention of each sequence, with the tolerances of test_prefix_gpu.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
from test_prefix_gpu import DEV, KINDS, Batch, lens_around

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    pk.kv_set_decode_workspace(None)


@pytest.mark.parametrize("kind", KINDS)
def test_plan_for_a_smaller_batch(kind):
    """The batch grew and the plan was not made anew: flagged, not used, and of the plan's buffer nothing is read past the
    header (the allocation goes on behind it with what would be wild indexes)."""
    rng = np.random.default_rng(3)
    small = Batch(71, kind, [(3000, lens_around(rng, 3000, 40, 100))], 8, 4, 128, 16)
    old, _ = small.plan()
    assert small.pieces(old) > 0
    b = Batch(73, kind, [(1600, lens_around(rng, 1600, 40, 100)) for _ in range(5)], 8, 4, 128, 16, width=small.width)
    Hq, H = b.dims()[:2]
    need = pk.kv_prefix_plan_bytes(len(b.lens), 5, Hq, H)
    assert need > old.numel()
    plan = torch.full((need,), 0x7F, dtype=torch.uint8, device=DEV)
    plan[:old.numel()] = old
    b.workspace(5)
    b.check(b.attend(plan, 5))
    assert pk.kv_get_device_error() == 64


@pytest.mark.parametrize("B,N,H,Hq,width", [(30, 2, 8, 32, 320), (30, 1, 8, 16, 320), (30, 1, 4, 32, 320), (30, 1, 8, 32, 321),
                                            (29, 1, 8, 32, 320)])
def test_plan_for_other_shapes(B, N, H, Hq, width):
    """Any one of the numbers that the plan was made for is another."""
    rng = np.random.default_rng(5)
    b = Batch(79, "fp8", [(4500, lens_around(rng, 4500, 30, 200))], 8, 4, 128, 16, width=320)
    tables = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    tables[:, :300] = torch.arange(300, device=DEV)
    lens = torch.full((B,), 4800, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, B] if N == 1 else [0, B // 2, B], dtype=torch.int32, device=DEV)
    room = max(pk.kv_prefix_plan_bytes(B, N, Hq, H), pk.kv_prefix_plan_bytes(30, 1, 32, 8))
    plan = torch.full((room,), 0x7F, dtype=torch.uint8, device=DEV)
    pk.kv_prefix_plan(plan, tables, lens, starts, width, B, N, Hq, H, 128, 16, 0, 0)
    assert b.pieces(plan) > 0
    b.workspace(1)
    b.check(b.attend(plan, 1))
    assert pk.kv_get_device_error() == 64
