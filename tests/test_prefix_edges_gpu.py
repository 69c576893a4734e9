"""Decodes over shared prefixes at the ends of what their documentation allows, against
64-bit attention of each sequence, with the tolerances of test_prefix_gpu.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
from test_prefix_gpu import DEV, KINDS, NAN_CODE, Batch, lens_around

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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("W,S", [(0, 0), (3500, 4), (200, 17)])
def test_length_past_its_table(kind, W, S):
    """A length past its table is cut to it in the shared part, in the own part and in the plan, and flagged."""
    rng = np.random.default_rng(W + 7)
    b = Batch(83, kind, [(4096, lens_around(rng, 4096, 24, 200) + [4352, 4352, 4000]), (4352, [4352] * 20)], 8, 4, 128, 16)
    assert b.width * 16 == 4352
    cut = list(b.lens)
    b.lens = [L + (int(rng.integers(1, 5000)) if L == 4352 else 0) for L in cut]
    b.lens[25] = 2 ** 31 - 1
    plan, N = b.plan(W, S)
    b.workspace(N)
    assert b.pieces(plan) > 0 or W == 200
    out = b.attend(plan, N, W, S)
    b.lens = cut
    b.check(out, W, S)
    assert pk.kv_get_device_error() == 2


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S", [0, 5, 40])
def test_plan_stays_while_a_window_moves(kind, S):
    """One plan under a window while lengths grow, until the windows of some, then of all members, have passed what they
    share, but for the sinks."""
    W = 2600
    rng = np.random.default_rng(S)
    final = [int(x) for x in rng.integers(7900, 8200, 40)] + [5300]
    b = Batch(89, kind, [(4800, final)], 4, 4, 128 if S else 64, 16)
    start = [4810 + int(x) for x in rng.integers(0, 30, 40)] + [4801]
    b.lens = start
    plan, N = b.plan(W, S)
    b.workspace(N)
    assert b.pieces(plan) > 0
    for step in (0.0, 0.1, 0.5, 0.8, 1.0):
        b.lens = [int(a + (f - a) * step) for a, f in zip(start, final)]
        b.check(b.attend(plan, N, W, S), W, S)
    assert min(b.lens[:40]) - W > 4800
    assert pk.kv_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_queries_of_a_fused_projection(kind):
    """Query rows at a stride larger than their heads."""
    rng = np.random.default_rng(11)
    b = Batch(97, kind, [(3000, lens_around(rng, 3000, 30, 100))], 8, 4, 128, 16)
    Hq, H, D, bs = b.dims()
    B, row = len(b.lens), (Hq + 2 * H) * D
    wide = torch.full((B, row), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :Hq * D] = b.q
    plan, N = b.plan()
    b.workspace(N)
    assert b.pieces(plan) > 0
    blk = tuple(b.scales) if kind == "fp8_block" else ()
    sc = {"fp8k": (b.k_scale,), "fp8": (b.k_scale, b.v_scale)}.get(kind, ())
    getattr(pk, f"paged_decode_attn_{kind}_prefix")(
        wide, *b.caches, *blk, b.out, torch.from_numpy(b.tables).to(DEV), torch.tensor(b.lens, dtype=torch.int32, device=DEV),
        plan, b.width, B, N, Hq, H, D, bs, D ** -0.5, *sc, row, 0, 0)
    b.check(b.out)


@pytest.mark.parametrize("members", [20, 50])  # 80 rows of a KV head, and 200 (two Q tiles)
@pytest.mark.parametrize("high", [-60, 0, 70, 100, 117])
def test_block_scales_over_their_range(members, high):
    """V scales of 2^-60 among blocks of 2^high, in the shared and in the own positions, and members whose blocks are of
    one kind: a key counts in the softmax sum whatever its V scale is."""
    rng = np.random.default_rng(high + 100)
    b = Batch(101 + high, "fp8_block", [(4000, lens_around(rng, 4000, members, 200)), (3000, lens_around(rng, 3000, members, 90))],
              4, 4, 128, 16)
    low = torch.from_numpy(rng.random(b.nb) < 0.5)
    low[torch.from_numpy(b.tables[0, :40].astype(np.int64))] = True  # the first pieces' tiles of one kind
    low[torch.from_numpy(b.tables[members, :30].astype(np.int64))] = False
    b.scales[1][:] = torch.where(low, 2.0 ** -60, 2.0 ** high).to(DEV)[:, None]
    out, pieces = b.run()
    assert pieces > 0
    b.check(out)
    assert pk.kv_get_device_error() == 0


@pytest.mark.parametrize("kind,members", [("bf16", 20), ("fp8k", 50)])
@pytest.mark.parametrize("size", [2.0 ** -9, 2.0 ** -10, 2.0 ** -16])
def test_small_values(kind, members, size):
    """BF16 V of shared positions is held exactly from 2^-9 up and within 2^-17 below, so rows are off by no more, whatever
    the size of V; from 2^-9 up the weights' rounding is all there is."""
    rng = np.random.default_rng(13)
    b = Batch(103, kind, [(4000, lens_around(rng, 4000, members, 100))], 4, 4, 128, 16)
    v = b.caches[1]
    v.copy_(torch.sign(v.float()) * size * (1 + 0.99 * torch.rand(v.shape, device=DEV)))  # [size, 2 size), NaN where it was
    out, pieces = b.run()
    assert pieces > 0
    b.check(out)
    for s in range(0, members, 7):
        k, x = b.values(s)
        z = torch.einsum("hgd,phd->hgp", b.q[s].double().view(4, 4, 128), k) * 128 ** -0.5
        w = torch.softmax(z, -1)
        want = torch.einsum("hgp,phd->hgd", w, x)
        zabs = torch.einsum("hgd,phd->hgp", b.q[s].double().view(4, 4, 128).abs(), k.abs()).amax(-1) * 128 ** -0.5
        n = k.shape[0]
        rel = torch.exp((128 + 8) * 2.0 ** -23 * zabs) - 1 + 2.0 ** -11 + 2.0 ** -19 + n * (2.0 ** -31 + 2.0 ** -23)
        tol = 2 * x.abs().amax() * rel + (0 if size >= 2.0 ** -9 else 2.0 ** -17)
        err = (out[s].double().view(want.shape) - want).abs() - want.abs() * 2.0 ** -8
        assert (err - tol[..., None]).max() <= 0, s


@pytest.mark.parametrize("kind", KINDS)
def test_values_that_are_not_finite(kind):
    """A shared V row that is not finite makes the rows that attend it non-finite, and may reach the rest of its group;
    members that attend alone keep theirs."""
    rng = np.random.default_rng(15)
    short = [1500, 2000, 700, 0]
    b = Batch(107, kind, [(4000, lens_around(rng, 4000, 30, 100) + short), (3000, lens_around(rng, 3000, 30, 100))], 8, 4, 128, 16)
    b.caches[1][int(b.tables[0, 200]), 5, :, 3] = NAN_CODE if b.caches[1].dtype == torch.uint8 else float("inf")  # position 3205
    out, pieces = b.run()
    assert pieces > 0
    assert not torch.isfinite(out[:30, :, 3].float()).any()
    assert (out[33] == 0).all()
    b.check(out, only=range(34, 64))
    # the short ones out of the group: their own rows alone
    out, pieces = b.run(starts=[0, 30, 34, 64])
    assert pieces > 0
    assert not torch.isfinite(out[:30, :, 3].float()).any()
    b.check(out, only=range(30, 64))
    assert pk.kv_get_device_error() == 0


@pytest.mark.parametrize("kind", ["fp8k", "fp8"])
@pytest.mark.parametrize("k_scale", [2.0 ** -140, 2.0 ** -100, 30.0])
def test_key_scales_small_and_large(kind, k_scale):
    """Scores that are all but equal, and scores far apart."""
    rng = np.random.default_rng(17)
    b = Batch(109, kind, [(3000, lens_around(rng, 3000, 30, 100))], 8, 4, 64, 16)
    b.k_scale = k_scale
    out, pieces = b.run()
    assert pieces > 0
    b.check(out)
