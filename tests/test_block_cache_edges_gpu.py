"""The block-scaled cache and the prefills at the ends of their ranges, against the plain
64-bit references, with the tolerances of test_block_cache_gpu.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
import reference64 as ref
from test_block_cache_gpu import DEV, KINDS, Pool, bf16, call, check_rows, f64, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    pk.kv_set_decode_workspace(None)


def rescale(pool, i, lens, scales, zero=None):
    """Give K (i = 0) or V (i = 1) of a block-scaled pool without a window the scales [blocks, heads], and zero codes
    in the blocks of `zero`; the reference's rows follow."""
    codes = pool.raw[i].cpu().numpy()
    if zero is not None:
        codes[zero] = 0
    pool.raw[i] = torch.from_numpy(codes).to(DEV)
    pool.scales[i][:] = scales
    for s, L in enumerate(lens):
        pos = np.arange(int(L))
        b = pool.tables[s, pos // pool.bs]
        pool.rows[i][s] = ref.e4m3_values(codes[b, pos % pool.bs]) * pool.scales[i][b].astype(np.float64)[..., None]


@pytest.mark.parametrize("small", ["zero", "nonzero"])
@pytest.mark.parametrize("high", [0, 70, 100, 117])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_block_scales_far_apart(form, D, high, small):
    """Blocks with V scales of 2^-60 (those that the write gives a block of zeros) among blocks of 2^high, in either
    order and for rows that see one kind only: a key counts in the softmax sum whatever its V scale is."""
    rng = np.random.default_rng(high + D)
    lens = np.array([200, 64, 700, 16, 150])
    new = np.ones(5, np.int64) if form == "decode" else np.array([200, 64, 30, 16, 150])
    pool = Pool(rng, "fp8_block", lens, lens, 2, D, 16, 0, 0)
    low = rng.random(pool.scales[1].shape[0]) < 0.5
    low[pool.tables[0, :4]], low[pool.tables[4, :5]] = True, False       # a row's first blocks of one kind
    rescale(pool, 1, lens, np.where(low[:, None], 2.0 ** -60, 2.0 ** high), low if small == "zero" else None)
    T = int(new.sum())
    q = bf16(rng.standard_normal((T, 4 * D)) * 0.3).to(DEV)
    out = torch.empty((T, 4, D), device=DEV, dtype=torch.float32 if form == "decode" else torch.bfloat16)
    call(pool, form, q, out, lens, np.concatenate([[0], np.cumsum(new)]), 4, 0, 0)
    check_rows(pool, form, q, out, lens, new, 4, 0, 0)
    assert pk.kv_get_device_error() == 0


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("D,k_exp,q_exp,isd_exp", [(64, 110, -116, -3), (64, 120, -114, -14), (128, 120, -114, -14)])
def test_small_queries_against_large_key_scales(form, D, k_exp, q_exp, isd_exp):
    """Scores of a few units from queries near the smallest numbers and K scales up to the largest: the product of the
    row's scale and the block's is in range where the row's alone is not."""
    rng = np.random.default_rng(D - q_exp)
    lens = np.array([200, 64, 300])
    new = np.ones(3, np.int64) if form == "decode" else np.array([40, 64, 5])
    pool = Pool(rng, "fp8_block", lens, lens, 2, D, 16, 0, 0)
    rescale(pool, 0, lens, 2.0 ** k_exp)
    T, isd = int(new.sum()), 2.0 ** isd_exp
    q = bf16(rng.standard_normal((T, 4 * D)) * 2.0 ** q_exp).to(DEV)
    out = torch.empty((T, 4, D), device=DEV, dtype=torch.float32 if form == "decode" else torch.bfloat16)
    args = [q, *pool.args(), out, i32(pool.tables), i32(lens)]
    geo = [4, 2, D, 16, isd, 4 * D, 0, 0]
    if form == "decode":
        pk.paged_decode_attn_fp8_block(*args, pool.tables.shape[1], 3, *geo)
    else:
        pk.paged_prefill_attn_fp8_block(*args, i32(np.concatenate([[0], np.cumsum(new)])), pool.tables.shape[1], 3, T, *geo)
    # (the check's scores are scaled by D^-1/2: the rest of isd is taken into its queries)
    check_rows(pool, form, q.double() * (isd * D ** 0.5), out, lens, new, 4, 0, 0)


@pytest.mark.parametrize("split", [False, True])
def test_decode_of_the_largest_scale(split):
    """V values of 2^120 and up, all positive: the sums before the division by the softmax's stay finite, in one piece
    and in many."""
    rng = np.random.default_rng(6)
    lens, H, D, bs = np.array([3000, 900]), 2, 128, 16
    pool = Pool(rng, "fp8_block", lens, lens, H, D, bs, 0, 0)
    pool.raw[1] = torch.from_numpy(ref.e4m3_codes(rng.uniform(1, 30, tuple(pool.raw[1].shape)))).to(DEV)
    rescale(pool, 1, lens, 2.0 ** 120)
    ws = torch.empty(pk.kv_decode_workspace_bytes(pool.tables.shape[1], 2, 4, H, D, bs), dtype=torch.uint8,
                     device=DEV) if split else None
    pk.kv_set_decode_workspace(ws)
    q = bf16(rng.standard_normal((2, 4 * D)) * 0.3).to(DEV)
    out = torch.empty((2, 4, D), device=DEV)
    call(pool, "decode", q, out, lens, None, 4, 0, 0)
    check_rows(pool, "decode", q, out, lens, np.ones(2, np.int64), 4, 0, 0)
    pk.kv_set_decode_workspace(None)


@pytest.mark.parametrize("isd,q_exp,k_exp", [(None, -120, -40), (0.0, 0, None), (1e-38, 0, -20)])
@pytest.mark.parametrize("kind", ["bf16", "fp8k", "fp8"])
def test_prefill_of_scores_that_vanish(kind, isd, q_exp, k_exp):
    """The prefills with float rows, where the score scale is zero or falls below the smallest number: every attended
    position has the same weight, and a masked one has none."""
    rng = np.random.default_rng(23)
    lens, new, H, Hq, D, bs = np.array([200, 64, 300]), np.array([40, 64, 5]), 2, 4, 128, 16
    pool = Pool(rng, kind, lens, new, H, D, bs, 0, 0)
    if k_exp is not None:
        pool.k_scale = 2.0 ** k_exp
    T = int(new.sum())
    q = bf16(rng.standard_normal((T, Hq * D)) * 2.0 ** q_exp).to(DEV)
    for W in (0, 30):
        out = torch.full((T, Hq, D), float("nan"), device=DEV)
        getattr(pk, f"paged_prefill_attn_{kind}")(
            q, *pool.raw, out, i32(pool.tables), i32(lens), i32(np.concatenate([[0], np.cumsum(new)])),
            pool.tables.shape[1], 3, T, Hq, H, D, bs, D ** -0.5 if isd is None else isd, *pool.scalars(), Hq * D, W)
        check_rows(pool, "prefill", torch.zeros_like(q), out, lens, new, Hq, W, 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,D,Hq,H,W,S", [(33, 64, 4, 2, 0, 0), (70, 128, 4, 1, 40, 5), (120, 64, 6, 2, 100, 17)])
def test_prefill_of_many_sequences(kind, B, D, Hq, H, W, S):
    """More sequences than a warp has lanes, their lengths spread over many length classes, empty ones and ones without
    new tokens among them: every item is found by its class."""
    rng = np.random.default_rng(B + D)
    lens = np.exp(rng.uniform(0, np.log(1500), B)).astype(np.int64)
    new = np.minimum(lens, rng.integers(0, 9, B))
    lens[::11], new[::11] = 0, 0
    new[5] = lens[5] = 300                                     # two items for each KV head
    pool = Pool(rng, kind, lens, new, H, D, 16, W, S)
    T = int(new.sum())
    q = bf16(rng.standard_normal((T, Hq * D))).to(DEV)
    out = torch.full((T, Hq, D), float("nan"), device=DEV, dtype=torch.bfloat16)
    call(pool, "prefill", q, out, lens, np.concatenate([[0], np.cumsum(new)]), Hq, W, S)
    check_rows(pool, "prefill", q, out, lens, new, Hq, W, S)
    assert pk.kv_get_device_error() == 0


@pytest.mark.parametrize("W,S", [(0, 0), (300, 20), (33, 200)])
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_block_scales_drawn_over_the_whole_range(form, W, S):
    """V scales from 2^-60 to 2^118, many not powers of two, over sequences of many tiles under windows and sinks: each
    row is as exact as its own largest value allows."""
    rng = np.random.default_rng(W + S + 1)
    lens = np.array([3000, 1333, 40])
    new = np.ones(3, np.int64) if form == "decode" else np.array([90, 7, 40])
    pool = Pool(rng, "fp8_block", lens, new, 2, 128, 16, W, S)
    live = np.isfinite(pool.scales[1])
    pool.scales[1][live] = (2.0 ** rng.integers(-60, 118, int(live.sum())) * rng.choice([1.0, 1.37, 1.91], int(live.sum()))
                            ).astype(np.float32)
    codes = pool.raw[1].cpu().numpy()
    for s, L in enumerate(lens):
        pos = np.arange(int(L))
        b = pool.tables[s, pos // 16]
        pool.rows[1][s] = ref.e4m3_values(codes[b, pos % 16]) * pool.scales[1][b].astype(np.float64)[..., None]
    T = int(new.sum())
    q = bf16(rng.standard_normal((T, 4 * 128)) * rng.choice([0.3, 3.0, 20.0], (T, 1))).to(DEV)
    ws = torch.empty(pk.kv_decode_workspace_bytes(pool.tables.shape[1], 3, 4, 2, 128, 16), dtype=torch.uint8, device=DEV)
    for split in (False, True) if form == "decode" else (False,):
        pk.kv_set_decode_workspace(ws if split else None)
        out = torch.empty((T, 4, 128), device=DEV, dtype=torch.float32 if form == "decode" else torch.bfloat16)
        call(pool, form, q, out, lens, np.concatenate([[0], np.cumsum(new)]), 4, W, S)
        check_rows(pool, form, q, out, lens, new, 4, W, S)
    pk.kv_set_decode_workspace(None)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_in_a_captured_graph(kind):
    """Captured once on a stream of its own, replayed with other queries and with the same tokens cut into other
    sequences' chunks."""
    rng = np.random.default_rng(29)
    lens, Hq, H, D, bs, W, S, T = np.array([200, 64, 300]), 4, 2, 128, 16, 50, 3, 80
    pool = Pool(rng, kind, lens, lens, H, D, bs, W, S)
    q = torch.zeros((T, Hq * D), device=DEV, dtype=torch.bfloat16)
    out = torch.zeros((T, Hq, D), device=DEV, dtype=torch.bfloat16)
    tables, d_lens, d_qsl, cache = i32(pool.tables), i32(lens), i32([0, 40, 60, 80]), pool.args()
    name = f"paged_prefill_attn_{kind}" + ("" if kind == "fp8_block" else "_sinks")

    def run():
        getattr(pk, name)(q, *cache, out, tables, d_lens, d_qsl, pool.tables.shape[1], 3, T, Hq, H, D, bs, D ** -0.5,
                          *pool.scalars(), Hq * D, W, S)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for new in ([40, 20, 20], [0, 64, 16], [79, 1, 0]):
        q.copy_(bf16(rng.standard_normal((T, Hq * D))))
        d_qsl.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        out.fill_(float("nan"))
        graph.replay()
        check_rows(pool, "prefill", q, out, lens, np.array(new), Hq, W, S)
    assert pk.kv_get_device_error() == 0
