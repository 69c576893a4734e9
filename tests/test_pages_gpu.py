"""The page calls on the GPU against plain references (reference64.py): whole
numbers, compared for equality; and the calls of a server together."""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
import reference64 as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV = torch.device("cuda")
BIT_RANGE, BIT_FULL = 16, 32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    pk.kv_set_decode_workspace(None)


def i32(x) -> torch.Tensor:
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def same(t: torch.Tensor, want, what=""):
    got = t.cpu().numpy()
    assert np.array_equal(got, np.asarray(want)), (what, got, want)


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("num_pairs", [1, 2, 33, 700])
def test_copy_blocks_of_every_width(num_pairs):
    """Pools of large and small blocks, in units of 16, 4 and 1 bytes, from bases on and off a 16-byte boundary, with
    padding pairs."""
    rng = np.random.default_rng(num_pairs)
    nb = 2 * num_pairs + 5
    perm = rng.permutation(nb)
    src, dst = perm[:num_pairs].astype(np.int32), perm[num_pairs:2 * num_pairs].astype(np.int32)
    if num_pairs > 2:
        src[::7] = -1
        dst[3::11] = -2
    pools, want = [], []
    for size, off in [(32768, 0), (2048, 0), (2032, 0), (16400, 0), (16, 0), (12, 0), (4096, 4), (7, 0), (50, 1),
                      (20000, 8)]:
        flat = torch.from_numpy(rng.integers(0, 256, nb * size + off, dtype=np.uint8)).to(DEV)
        pools.append(flat[off:].view(nb, size))
        w = pools[-1].cpu().numpy().copy()
        ok = (src >= 0) & (dst >= 0)
        w[dst[ok]] = w[src[ok]]
        want.append(w)
    pk.kv_copy_blocks(pools, i32(src), i32(dst), num_pairs, nb)
    for i, (p, w) in enumerate(zip(pools, want)):
        same(p, w, i)
    assert pk.kv_get_device_error() == 0


def test_copy_blocks_many_pools_and_ids_out_of_range():
    rng = np.random.default_rng(1)
    nb, n = 9, 300                                            # more pools than one launch takes
    data = torch.from_numpy(rng.integers(0, 256, (n, nb, 2048), dtype=np.uint8)).to(DEV)
    want = data.cpu().numpy().copy()
    want[:, 7] = want[:, 2]
    pk.kv_copy_blocks(list(data.unbind(0)), i32([2, 9, 1, -1]), i32([7, 3, 1 << 30, 4]), 4, nb)
    same(data, want)
    assert pk.kv_get_device_error() == BIT_RANGE
    with pytest.raises(ValueError, match="equal blocks"):
        pk.kv_copy_blocks([data], i32([0]), i32([1]), 1, 7)
    pk.kv_copy_blocks([], i32([0]), i32([1]), 1, 7)


# ---------------------------------------------------------------------------
def random_state(rng, B, width, nb, bs, share=0.3):
    """Tables of rows with random lengths, some blocks shared between rows, some entries given back, and the counts."""
    tables = np.full((B, width), -1, np.int32)
    refs = np.zeros(nb, np.int32)
    free = list(rng.permutation(nb))
    lens = np.zeros(B, np.int32)
    for s in range(B):
        L = int(rng.integers(0, width * bs + 1))
        for j in range(-(-L // bs)):
            others = tables[:s][tables[:s] >= 0]
            if others.size and rng.random() < share:
                tables[s, j] = rng.choice(others)
            elif free:
                tables[s, j] = free.pop()
            else:
                break
            refs[tables[s, j]] += 1
            lens[s] = min(L, (j + 1) * bs)
    return tables, refs, lens


@pytest.mark.parametrize("B,width,nb,bs", [(1, 1, 1, 16), (5, 7, 30, 16), (40, 20, 700, 32), (3, 300, 900, 16)])
def test_free_blocks(B, width, nb, bs):
    rng = np.random.default_rng(B)
    tables, refs, lens = random_state(rng, B, width, nb, bs)
    first = rng.integers(-2, width + 1, B).astype(np.int32)
    end = (first + rng.integers(-1, width + 2, B)).astype(np.int32)
    t, r = i32(tables), i32(refs)
    pk.kv_free_blocks(t, r, i32(first), i32(end), width, B, nb)
    ref.free_blocks(tables, refs, first, end)
    same(t, tables), same(r, refs)
    # what a window with sinks leaves behind
    for W, S in ((1, 0), (bs + 3, 1), (2 * bs, bs), (40, 5 * bs), (10 ** 6, 0), (0, 4)):
        f = np.full(B, -(-S // bs))
        e = np.maximum(lens.astype(np.int64) - W, 0) // bs if W else np.zeros(B)
        pk.kv_free_window_blocks(t, r, i32(lens), width, B, nb, bs, W, S)
        ref.free_blocks(tables, refs, f, e)
        same(t, tables, (W, S)), same(r, refs, (W, S))
    assert pk.kv_get_device_error() == 0


def test_free_blocks_flags_what_is_out_of_range():
    t, r = i32([[0, 1, 5, -1], [1, 2, 2, -1]]), i32([1, 1, 1, 0, 7])
    pk.kv_free_blocks(t, r, i32([0, 0]), i32([4, 4]), 4, 2, 5)
    same(t, np.full((2, 4), -1)), same(r, [0, 0, 0, 0, 7])     # 1 and 2 are freed twice, 5 is no block
    assert pk.kv_get_device_error() == BIT_RANGE


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,width,nb,bs,forks", [(2, 1, 3, 16, 1), (12, 9, 200, 16, 6), (90, 30, 4000, 64, 45),
                                                 (3000, 3, 40001, 16, 1500), (40, 40, 60000, 32, 20)])
def test_fork_blocks(B, width, nb, bs, forks):
    rng = np.random.default_rng(B + 1)
    tables, refs, lens = random_state(rng, B, width, nb, bs)
    rows = rng.permutation(B)
    dst = rows[:forks].astype(np.int32)
    src = rng.choice(rows[forks:], forks).astype(np.int32)
    whole = np.zeros(B, np.int64)
    whole[dst] = width
    ref.free_blocks(tables, refs, np.zeros(B), whole)
    if width > 4:                                             # a parent whose window has left pages behind
        gone = np.zeros(B, np.int64)
        gone[src[0]] = 2
        ref.free_blocks(tables, refs, np.zeros(B), gone)
    if nb == 40001:                                           # the free blocks are the last ones
        used = refs[:nb - 2 * forks] == 0
        refs[:nb - 2 * forks][used] = 1
    t, r, n = i32(tables), i32(refs), i32(lens)
    cs, cd = torch.full((forks,), 9, device=DEV, dtype=torch.int32), torch.full((forks,), 9, device=DEV, dtype=torch.int32)
    pk.kv_fork_blocks(t, n, r, i32(src), i32(dst), cs, cd, forks, width, B, nb, bs)
    want = ref.fork_blocks(tables, lens, refs, src, dst, bs)
    same(cs, want[0], "src"), same(cd, want[1], "dst"), same(t, tables), same(r, refs), same(n, lens)
    assert pk.kv_get_device_error() == 0


def test_fork_blocks_refuses_what_cannot_be_made():
    bs = 16
    tables = np.array([[0, 1, -1], [2, -1, -1], [-1, -1, -1], [-1, -1, -1], [3, 4, 5], [-1, -1, -1], [8, -1, -1]], np.int32)
    lens = np.array([20, 16, 0, 0, 48, 49, 3], np.int32)      # row 5's length is past its table, row 6's block past the pool
    refs = np.array([1, 1, 1, 1, 1, 1, 0, 0], np.int32)
    for src, dst, bits in [([0, 0], [2, 2], BIT_RANGE),       # a row twice
                           ([0, 2], [2, 3], BIT_RANGE),       # a row written and read
                           ([0, 0, 9], [-1, 7, 2], BIT_RANGE),
                           ([5, 6], [2, 3], BIT_RANGE),
                           ([2], [2], BIT_RANGE),
                           ([0, 1, 0, 0], [2, 3, 5, 6], BIT_FULL)]:  # two free blocks for three partial pages
        t, r, n = i32(tables), i32(refs), i32(lens)
        cs, cd = torch.empty(len(src), device=DEV, dtype=torch.int32), torch.empty(len(src), device=DEV, dtype=torch.int32)
        pk.kv_fork_blocks(t, n, r, i32(src), i32(dst), cs, cd, len(src), 3, 7, 8, bs)
        tt, rr, nn = tables.copy(), refs.copy(), lens.copy()
        want = ref.fork_blocks(tt, nn, rr, src, dst, bs)
        same(cs, want[0]), same(cd, want[1]), same(t, tt), same(r, rr), same(n, nn)
        assert pk.kv_get_device_error() == bits, (src, dst)


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,width,nb,used", [(1, 1, 1, 0), (1, 1, 1, 1), (3, 4, 2, 1), (4, 9, 33, 20), (4, 9, 31, 31),
                                             (30, 40, 1000, 333), (50, 100, 5000, 2600), (2, 70, 40000, 100),
                                             (64, 700, 50001, 41000), (5, 5, 64, 0)])
def test_compact_blocks(B, width, nb, used, in_place):
    rng = np.random.default_rng(nb + used)
    ids = rng.permutation(nb)[:used].astype(np.int32)
    tables = np.full(B * width, -1, np.int32)
    refs = np.zeros(nb, np.int32)
    at = rng.permutation(B * width)[:min(used, B * width)]
    tables[at] = ids[:at.size]
    refs[ids] = 1                                             # (blocks that no table names may be in use)
    for e in np.flatnonzero(tables < 0)[::5]:                 # some shared
        if used:
            tables[e] = rng.choice(ids)
            refs[tables[e]] += 1
    tables = tables.reshape(B, width)
    t, r = i32(tables), i32(refs)
    nt, nr = (t, r) if in_place else (torch.full_like(t, 99), torch.full_like(r, 99))
    new_ids = torch.full((nb,), 99, device=DEV, dtype=torch.int32)
    cs, cd = (torch.full((max(nb // 2, 1),), 99, device=DEV, dtype=torch.int32) for _ in range(2))
    count = torch.full((1,), 99, device=DEV, dtype=torch.int32)
    pk.kv_compact_blocks(t, r, nt, nr, new_ids, cs, cd, count, width, B, nb)
    wt, wr, wi, ws, wd, wu = ref.compact_blocks(tables, refs)
    same(count, [wu]), same(new_ids, wi), same(nr, wr), same(nt, wt)
    same(cs[:nb // 2], ws), same(cd[:nb // 2], wd)
    if not in_place:
        same(t, tables), same(r, refs)
    assert pk.kv_get_device_error() == 0


def test_compact_blocks_flags_entries_of_free_blocks():
    t, r = i32([[0, 3, 1, 7]]), i32([0, -2, 0, 1, 0])
    nt, nr, ids = torch.empty_like(t), torch.empty_like(r), torch.empty_like(r)
    cs, cd, n = i32([9, 9]), i32([9, 9]), i32([9])
    pk.kv_compact_blocks(t, r, nt, nr, ids, cs, cd, n, 4, 1, 5)
    same(nt, [[-1, 0, -1, -1]]), same(nr, [1, 0, 0, 0, 0]), same(ids, [-1, -1, -1, 0, -1])
    same(cs, [3, -1]), same(cd, [0, -1]), same(n, [1])
    assert pk.kv_get_device_error() == BIT_RANGE


# ---------------------------------------------------------------------------
def test_the_calls_together():
    """A server's steps on two layers: prompts written, a chunk attended, pages behind the window freed, each sequence
    forked, the forks appended to and decoded, the pool compacted, and decoded again. Every sequence's result is that
    of a cache of its own, and the compaction changes no bit."""
    rng = np.random.default_rng(17)
    H, Hq, D, bs, W, S, layers = 2, 4, 128, 16, 50, 4, 2
    nb, width, B = 160, 20, 6
    prompt = np.array([130, 16, 75])
    tables = np.full((B, width), -1, np.int32)
    refs = np.zeros(nb, np.int32)
    perm = rng.permutation(nb)
    at = 0
    lens = np.zeros(B, np.int32)
    for s, L in enumerate(prompt):
        n = -(-int(L) // bs)
        tables[s, :n] = perm[at:at + n]
        refs[perm[at:at + n]] = 1
        lens[s], at = L, at + n
    rows = lambda T: torch.randn((layers, 2, T, H * D), device=DEV).to(torch.bfloat16)  # noqa: E731
    torch.manual_seed(5)
    codes = torch.full((layers, 2, nb, bs, H, D), 0x7F, device=DEV, dtype=torch.uint8)
    scales = torch.full((layers, 2, nb, H), float("nan"), device=DEV)
    t, r, n = i32(tables), i32(refs), i32(lens)
    first = rows(int(prompt.sum()))
    qsl = i32(np.concatenate([[0], np.cumsum(prompt), [prompt.sum()] * 3]))
    T = int(prompt.sum())
    q = torch.randn((T, Hq * D), device=DEV).to(torch.bfloat16)
    chunk = torch.empty((layers, T, Hq, D), device=DEV, dtype=torch.bfloat16)

    def write(x, lens, qsl, T):
        for l in range(layers):
            pk.kv_write_fp8_block(x[l, 0], x[l, 1], codes[l, 0], codes[l, 1], scales[l, 0], scales[l, 1], t, lens, qsl,
                                  width, B, T, H, D, bs, H * D, H * D)

    def decode(qd):
        out = torch.empty((layers, B, Hq, D), device=DEV)
        for l in range(layers):
            pk.paged_decode_attn_fp8_block(qd, codes[l, 0], codes[l, 1], scales[l, 0], scales[l, 1], out[l], t, n, width,
                                           B, Hq, H, D, bs, D ** -0.5, Hq * D, W, S)
        return out
    write(first, n, qsl, T)
    for l in range(layers):
        pk.paged_prefill_attn_fp8_block(q, codes[l, 0], codes[l, 1], scales[l, 0], scales[l, 1], chunk[l], t, n, qsl, width,
                                        B, T, Hq, H, D, bs, D ** -0.5, Hq * D, W, S)
    values = lambda l, i, blocks, pos: (ref.e4m3_values(codes[l, i].cpu().numpy()[blocks, pos % bs])  # noqa: E731
                                        * scales[l, i].cpu().numpy()[blocks].astype(np.float64)[..., None])
    # the chunk against the definition over the values that the cache holds
    for l in range(layers):
        row = 0
        for s, L in enumerate(prompt):
            pos = np.arange(L)
            k, v = (values(l, i, tables[s, pos // bs], pos) for i in range(2))
            for P in range(L):
                for h in range(Hq):
                    o, vmax, _ = ref.attention(q[row].double().cpu().numpy()[h * D:(h + 1) * D], k[:, h // 2], v[:, h // 2],
                                               P, W, S, D ** -0.5)
                    err = np.abs(chunk[l, row, h].double().cpu().numpy() - o)
                    assert (err <= np.abs(o) * 2.0 ** -8 + 2 * vmax * 2.0 ** -10).all()   # the f16 weights' 2^-11, doubled
                row += 1
    # pages behind the window go, every sequence is forked, the forks' partial pages are copied
    pk.kv_free_window_blocks(t, r, n, width, B, nb, bs, W, S)
    cs, cd = torch.empty(3, device=DEV, dtype=torch.int32), torch.empty(3, device=DEV, dtype=torch.int32)
    pk.kv_fork_blocks(t, n, r, i32([0, 1, 2]), i32([3, 4, 5]), cs, cd, 3, width, B, nb, bs)
    pools = [p for l in range(layers) for p in (codes[l, 0], codes[l, 1], scales[l, 0], scales[l, 1])]
    pk.kv_copy_blocks(pools, cs, cd, 3, nb)
    torch.cuda.synchronize()
    assert cs.tolist()[1] == -1 and cs.tolist()[0] >= 0
    # a new token each (the row at 16 positions starts a block: given by hand, as a server's allocator does)
    lens2 = np.concatenate([prompt, prompt]) + 1
    tables, refs = t.cpu().numpy(), r.cpu().numpy()
    for s in (1, 4):
        b = int(np.flatnonzero(refs == 0)[0])
        tables[s, 1], refs[b] = b, 1
    t.copy_(i32(tables)), r.copy_(i32(refs)), n.copy_(i32(lens2))
    second = rows(B)
    write(second, n, i32(np.arange(B + 1)), B)
    qd = torch.randn((B, Hq * D), device=DEV).to(torch.bfloat16)
    before = decode(qd)
    for l in range(layers):
        for s in range(B):
            pos = np.arange(lens2[s])
            blocks = tables[s, pos // bs]
            blocks = np.where(blocks < 0, 0, blocks)          # given back: not attended
            k, v = (values(l, i, blocks, pos) for i in range(2))
            for h in range(Hq):
                o, vmax, zabs = ref.attention(qd[s].double().cpu().numpy()[h * D:(h + 1) * D], k[:, h // 2], v[:, h // 2],
                                              int(lens2[s]) - 1, W, S, D ** -0.5)
                err = np.abs(before[l, s, h].double().cpu().numpy() - o)
                assert (err <= 2 * vmax * (136 * 2.0 ** -23 * zabs * 1.01 + 2.0 ** -16)).all()
    # the pool is compacted; the same tokens are attended at other places
    nt, nr, ids = torch.empty_like(t), torch.empty_like(r), torch.empty_like(r)
    ms, md, used = (torch.empty(k, device=DEV, dtype=torch.int32) for k in (nb // 2, nb // 2, 1))
    pk.kv_compact_blocks(t, r, nt, nr, ids, ms, md, used, width, B, nb)
    pk.kv_copy_blocks(pools, ms, md, nb // 2, nb)
    u = int(used)
    assert u == int((refs > 0).sum()) and int((ms >= 0).sum()) > 0
    assert bool((nr[:u] > 0).all()) and bool((nr[u:] == 0).all())
    codes[:, :, u:] = 0x7F
    t.copy_(nt)
    assert torch.equal(decode(qd), before)
    assert pk.kv_get_device_error() == 0


def test_page_calls_in_a_captured_graph():
    """A fork with its page copy, a release and a compaction with its copy captured once (on a stream of its own),
    replayed over three other states that are put into the same buffers."""
    rng = np.random.default_rng(31)
    B, width, nb, bs, forks, size = 40, 9, 400, 16, 12, 4096
    t, lens, refs = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((B, width), (B,), (nb,)))
    src, dst, first, end = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (forks, forks, B, B))
    cs, cd = (torch.zeros(forks, dtype=torch.int32, device=DEV) for _ in range(2))
    nt, nr, ids, num = torch.zeros_like(t), torch.zeros_like(refs), torch.zeros_like(refs), torch.zeros_like(refs[:1])
    ms, md = (torch.zeros(nb // 2, dtype=torch.int32, device=DEV) for _ in range(2))
    pools = [torch.zeros((nb, n), dtype=torch.uint8, device=DEV) for n in (size, 32)]

    def run():
        pk.kv_fork_blocks(t, lens, refs, src, dst, cs, cd, forks, width, B, nb, bs)
        pk.kv_copy_blocks(pools, cs, cd, forks, nb)
        pk.kv_free_blocks(t, refs, first, end, width, B, nb)
        pk.kv_compact_blocks(t, refs, nt, nr, ids, ms, md, num, width, B, nb)
        pk.kv_copy_blocks(pools, ms, md, nb // 2, nb)

    run()
    assert pk.kv_get_device_error() == BIT_RANGE           # (forks of row 0 to itself, entries of free blocks)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        ht, hl, hr = np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(nb, np.int32)
        perm = rng.permutation(nb)
        for s in range(20):                                # rows 20.. are free
            hl[s] = rng.integers(0, width * bs + 1)
            n = -(-int(hl[s]) // bs)
            ht[s, :n], perm = perm[:n], perm[n:]
            hr[ht[s, :n]] = 1
        hs, hd = rng.integers(0, 20, forks).astype(np.int32), (20 + rng.permutation(20)[:forks]).astype(np.int32)
        hf, he = np.zeros(B, np.int32), np.zeros(B, np.int32)
        he[rng.permutation(20)[:8]] = width                # eight parents end
        data = [rng.integers(0, 256, p.shape, dtype=np.uint8) for p in pools]
        for dev, host in zip((t, lens, refs, src, dst, first, end, *pools), (ht, hl, hr, hs, hd, hf, he, *data)):
            dev.copy_(torch.from_numpy(host))
        graph.replay()
        ws, wd = ref.fork_blocks(ht, hl, hr, hs, hd, bs)
        for d in data:
            d[wd[wd >= 0]] = d[ws[ws >= 0]]
        ref.free_blocks(ht, hr, hf, he)
        wt, wr, wi, wms, wmd, used = ref.compact_blocks(ht, hr)
        for d in data:
            d[wmd[wmd >= 0]] = d[wms[wms >= 0]]
        for got, want, what in ((lens, hl, "lens"), (cs, ws, "src"), (cd, wd, "dst"), (t, ht, "tables"), (refs, hr, "refs"),
                                (nt, wt, "new tables"), (nr, wr, "new refs"), (ids, wi, "ids"), (ms, wms, "moves"),
                                (md, wmd, "to"), (num, [used], "used")):
            same(got, want, what)
        for p, d in zip(pools, data):
            live = wr > 0                                   # (a moved block's old place is free)
            same(p[torch.from_numpy(live).to(DEV)], d[live], "pool")
    assert pk.kv_get_device_error() == 0
