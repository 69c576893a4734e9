"""The block-scaled FP8 cache and attention with sinks on the GPU, against
plain 64-bit references (reference64.py).

The write is compared bit for bit. The attention tolerances are sums of the
roundings on the way, taken for each output row from its own data:
  scores    a D-term sum in 32 bits, each partial sum off by at most 2^-23 of
            the sum of magnitudes z_abs: dz = (D + 8) 2^-23 z_abs (and the scale,
            the running maximum and exp2's own 2^-22 in the 8 and below);
  weights   relative error e^dz - 1 + 2^-20 (exp2, the split into two f16
            parts, 2^-22, or three BF16 ones, 2^-26), or 2^-11 as one f16;
  sums      n positive terms in 32 bits, n 2^-24 relative;
  output    at most 2 max|v| times the relative errors of weights and sums, and
            half a step of BF16 (2^-8) where the rows are BF16.
The prefill holds BF16 V as f16 of v 2^-8 (2^-17 absolute below 2^-6) and
weights below 2^-21 of the largest as subnormals (n 2^-31 of max|v|).
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
import reference64 as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

DEV = torch.device("cuda")
NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    pk.kv_set_decode_workspace(None)


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def i32(x) -> torch.Tensor:
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def permuted_tables(rng, lens, bs, spare=3, extra=0):
    need = [-(-int(L) // bs) for L in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), max(max(need), 1) + extra), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    return tables, nb


# ---------------------------------------------------------------------------
# the block-scaled write
# ---------------------------------------------------------------------------
class Cache:
    """Poisoned code pools and scale pools on the GPU, and the same on the host."""

    def __init__(self, nb, bs, H, D, scale=np.nan):
        self.codes = [np.full((nb, bs, H, D), NAN_CODE, np.uint8) for _ in range(2)]
        self.scales = [np.full((nb, H), scale, np.float32) for _ in range(2)]
        self.upload()

    def upload(self):
        self.dc = [torch.from_numpy(c).to(DEV) for c in self.codes]
        self.ds = [torch.from_numpy(s).to(DEV) for s in self.scales]

    def check(self, what=""):
        for i in range(2):
            got, want = self.ds[i].cpu().numpy(), self.scales[i]
            assert np.array_equal(got, want, equal_nan=True), f"{what} scales {i}"
            got = self.dc[i].cpu().numpy()
            bad = np.flatnonzero(got.ravel() != self.codes[i].ravel())
            assert bad.size == 0, (what, i, bad[:8], got.ravel()[bad[:8]], self.codes[i].ravel()[bad[:8]])


def write_both(cache, key, value, tables, lens, qsl, H, D, bs, stream=None):
    T = key.shape[0]
    pk.kv_write_fp8_block(key.to(DEV), value.to(DEV), *cache.dc, *cache.ds, i32(tables), i32(lens), i32(qsl),
                          tables.shape[1], len(lens), T, H, D, bs, key.shape[1], value.shape[1], stream)
    ref.write_block(f64(key), f64(value), cache.codes, cache.scales, tables, lens, qsl, H, D, bs)


@pytest.mark.parametrize("D,bs,H,pad", [(64, 16, 2, 0), (128, 16, 3, 8), (128, 32, 1, 3), (128, 64, 8, 0),
                                        (256, 16, 2, 0), (256, 128, 1, 5), (64, 256, 2, 16), (256, 256, 1, 0),
                                        (128, 128, 2, 0), (128, 256, 1, 8), (64, 32, 5, 0)])
def test_write_block_bit_exact_over_appends(D, bs, H, pad):
    """Prompts, then chunks and single tokens of growing and shrinking magnitude: scales that grow, that stay, and
    blocks begun in the middle of a call."""
    rng = np.random.default_rng(D + bs + H)
    final = np.array([3 * bs + 5, 1, 2 * bs, bs + 1, 0, 40])
    tables, nb = permuted_tables(rng, final, bs)
    cache = Cache(nb, bs, H, D)
    lens = np.zeros_like(final)
    step = 0
    while (lens < final).any():
        most = [final // 2, np.full_like(final, 7), np.full_like(final, 1), np.full_like(final, bs + 3)][step % 4]
        new = np.minimum(final - lens, most) if step < 12 else final - lens
        lens = lens + new
        qsl = np.concatenate([[0], np.cumsum(new)])
        T = int(qsl[-1])
        size = 2.0 ** rng.integers(-6, 7, (max(T, 1), H, 1))
        x = [rng.standard_normal((T, H, D)) * size[:T] for _ in range(2)]
        key, value = (bf16(np.concatenate([a.reshape(T, H * D), rng.standard_normal((T, p))], 1))
                      for a, p in zip(x, (pad, pad + 8)))
        write_both(cache, key, value, tables, lens, qsl, H, D, bs)
        cache.check(f"step {step}")
        step += 1
    assert pk.kv_get_device_error() == 0


def test_write_block_values_at_the_edges():
    """Zeros, NaN, infinities, subnormals, the largest values, and |x| on either side of 448 times a power of two."""
    H, D, bs = 1, 64, 16
    rows = [np.zeros(D), np.full(D, np.nan), np.full(D, np.inf), np.full(D, -np.inf), np.full(D, 2.0 ** -133),
            np.full(D, 3.3e38), np.full(D, -2.0 ** -60), np.full(D, 448.0), np.full(D, 450.0), np.full(D, 7.0),
            np.full(D, 7.03125), np.full(D, 1.75 * 2.0 ** -60), np.linspace(-1, 1, D) * 2.0 ** -50]
    mixed = np.linspace(-3, 3, D)
    mixed[[0, 5, 9]] = [np.nan, np.inf, -np.inf]
    rows.append(mixed)
    n = len(rows)
    tables = np.arange(n, dtype=np.int32)[:, None]          # a block each, one token each
    cache = Cache(n, bs, H, D)
    write_both(cache, bf16(rows), bf16(rows[::-1]), tables, np.ones(n, np.int64), np.arange(n + 1), H, D, bs)
    cache.check("first tokens")
    # a second token: the scale grows from the smallest to the largest, or stays
    write_both(cache, bf16(rows[::-1]), bf16(rows), tables, np.full(n, 2), np.arange(n + 1), H, D, bs)
    cache.check("second tokens")


def test_write_block_leaves_what_is_not_its_own():
    """Padding blocks, empty sequences, positions below 0 and past the table, tokens in no sequence; bad layouts set
    their bits and write nothing of their sequence."""
    rng = np.random.default_rng(5)
    H, D, bs = 2, 128, 16
    lens = np.array([40, 0, 20, 70, 5])
    new = np.array([40, 0, 20, 30, 9])                       # the last: more tokens than positions
    tables = np.array([[3, -1, 0, -1], [-1] * 4, [5, 6, -1, -1], [7, 8, 9, 10], [2, -1, -1, -1]], np.int32)
    qsl = np.concatenate([[0], np.cumsum(new)])
    T = int(qsl[-1]) + 4                                     # four more rows than the sequences have
    key, value = bf16(rng.standard_normal((T, H * D))), bf16(rng.standard_normal((T, H * D)))
    cache = Cache(12, bs, H, D, scale=1.0)                   # length 70 is past the table's 64 positions
    write_both(cache, key, value, tables, lens, qsl, H, D, bs)
    cache.check("skips")
    assert pk.kv_get_device_error() == 2
    cache = Cache(12, bs, H, D, scale=1.0)
    for bad in ([0, 5, 3, 8, 9, 9], [0, -1, 3, 8, 9, 9], [0, 5, 5, 8, 9, T + 1]):
        pk.kv_write_fp8_block(key.to(DEV), value.to(DEV), *cache.dc, *cache.ds, i32(np.zeros((5, 4)) - 1), i32(lens * 0),
                              i32(bad), 4, 5, T, H, D, bs, H * D, H * D)
        assert pk.kv_get_device_error() == 4
    cache.check("bad layouts")


def test_write_block_many_sequences_and_streams():
    """1,500 sequences of one new token each (two rounds of the search), on a stream of its own, from rows that start
    off a 16-byte boundary."""
    rng = np.random.default_rng(11)
    H, D, bs, B = 1, 64, 16, 1500
    lens = rng.integers(1, 40, B)
    tables, nb = permuted_tables(rng, lens, bs)
    cache = Cache(nb, bs, H, D, scale=0.25)
    for c in cache.codes:
        c[:] = rng.integers(0, 127, c.shape)
    cache.upload()
    flat = bf16(rng.standard_normal(B * H * D + 1)).to(DEV)
    key = flat[1:].view(B, H * D)
    assert key.data_ptr() % 16
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    qsl = np.arange(B + 1)
    pk.kv_write_fp8_block(key, key, *cache.dc, *cache.ds, i32(tables), i32(lens), i32(qsl), tables.shape[1], B, B, H, D,
                          bs, H * D, H * D, stream)
    stream.synchronize()
    ref.write_block(f64(key), f64(key), cache.codes, cache.scales, tables, lens, qsl, H, D, bs)
    cache.check()


@pytest.mark.parametrize("D,bs,H", [(128, 64, 1), (128, 128, 1), (64, 256, 3), (256, 32, 1)])
def test_write_block_steps_with_nothing_to_write(D, bs, H):
    """2,000 sequences of a token or two, so that items with nothing to write stand between those of one CTA, by tasks
    of several warps, with scales that differ from block to block: no warp may take another step's maximum."""
    rng = np.random.default_rng(D + bs)
    B = 2000
    new = rng.integers(0, 3, B)
    lens = np.maximum(new, rng.integers(1, bs + 8, B))
    tables, nb = permuted_tables(rng, lens, bs)
    cache = Cache(nb, bs, H, D, scale=2.0 ** -20)
    for c in cache.codes:
        c[:] = rng.integers(0, 127, c.shape)
    cache.upload()
    T = int(new.sum())
    size = 2.0 ** rng.integers(-30, 31, (T, H, 1))
    key, value = (bf16((rng.standard_normal((T, H, D)) * size).reshape(T, H * D)) for _ in range(2))
    write_both(cache, key, value, tables, lens, np.concatenate([[0], np.cumsum(new)]), H, D, bs)
    cache.check()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
KINDS = ["bf16", "fp8k", "fp8", "fp8_block"]


class Pool:
    """A cache of `kind` filled with random rows at the attended positions and NaN everywhere else: rows past the end,
    spare blocks and their scales, and (where `given_back`) blocks whose table entries are -1."""

    def __init__(self, rng, kind, lens, new, H, D, bs, W, S, wide=False):
        self.kind, self.H, self.D, self.bs = kind, H, D, bs
        self.tables, nb = permuted_tables(rng, lens, bs)
        self.k_scale, self.v_scale = 0.031, 0.017
        k8, v8 = kind != "bf16", kind in ("fp8", "fp8_block")
        shape = (nb, bs, H, D)
        self.scales = None
        if kind == "fp8_block":
            low, high = (-24, 24) if wide else (-8, -4)
            self.scales = [(2.0 ** rng.integers(-8, -4, (nb, H)) * rng.choice([1.0, 1.37], (nb, H))).astype(np.float32),
                           (2.0 ** rng.integers(low, high, (nb, H)) * rng.choice([1.0, 1.91], (nb, H))).astype(np.float32)]
        raw, vals = [], []
        for i, e4m3 in enumerate((k8, v8)):
            x = rng.standard_normal(shape)
            if e4m3:
                c = ref.e4m3_codes(x * 40)
                v = ref.e4m3_values(c)
                v = v * (self.scales[i][:, None, :, None].astype(np.float64) if self.scales
                         else float(np.float32((self.k_scale, self.v_scale)[i])))
                raw.append(torch.from_numpy(c))
            else:
                t = bf16(x)
                v = f64(t)
                raw.append(t)
            vals.append(v)
        keep = np.zeros((nb, bs), bool)
        rows = [[], []]
        for s, L in enumerate(lens):
            L, n = int(L), int(new[s])
            lo = max(0, L - n + 1 - W) if W else 0
            pos = np.arange(L)
            b = self.tables[s, pos // bs] if L else np.zeros(0, int)
            for i in range(2):
                rows[i].append(vals[i][b, pos % bs])        # [L, H, D]
            live = (pos >= lo) | (pos < S)
            keep[b[live], pos[live] % bs] = True
            first = -(-min(S, lo) // bs)
            self.tables[s, first:max(first, lo // bs)] = -1
        for t in raw:
            t[torch.from_numpy(~keep)] = NAN_CODE if t.dtype == torch.uint8 else float("nan")
        if self.scales:
            for sc in self.scales:
                sc[~keep.any(1)] = np.nan
        self.rows = rows
        self.raw = [t.to(DEV) for t in raw]

    def args(self):
        extra = [torch.from_numpy(s).to(DEV) for s in self.scales] if self.scales else []
        return self.raw + extra

    def scalars(self):
        return {"bf16": [], "fp8k": [self.k_scale], "fp8": [self.k_scale, self.v_scale], "fp8_block": []}[self.kind]


def call(pool, form, q, out, lens, qsl, Hq, W, S, q_stride=None, stream=None):
    H, D, bs = pool.H, pool.D, pool.bs
    name = f"paged_{form}_attn_{pool.kind}" + ("" if pool.kind == "fp8_block" else "_sinks")
    meta = [i32(pool.tables), i32(lens)] + ([i32(qsl)] if form == "prefill" else [])
    geo = [pool.tables.shape[1], len(lens)] + ([q.shape[0]] if form == "prefill" else []) + [Hq, H, D, bs, D ** -0.5]
    getattr(pk, name)(q, *pool.args(), out, *meta, *geo, *pool.scalars(), q_stride or Hq * D, W, S, stream)


def check_rows(pool, form, q, out, lens, new, Hq, W, S):
    H, D, g = pool.H, pool.D, Hq // pool.H
    got, qd = f64(out), f64(q)[:, :Hq * D].reshape(-1, Hq, D)
    assert np.isfinite(got).all()
    row = 0
    for s, L in enumerate(lens):
        for j in range(int(new[s])):
            P = int(L) - int(new[s]) + j
            for h in range(Hq):
                o, vmax, zabs = ref.attention(qd[row, h], pool.rows[0][s][:, h // g], pool.rows[1][s][:, h // g], P, W, S,
                                              D ** -0.5)
                n = max(P + 1, 0)
                dz = (D + 8) * 2.0 ** -23 * zabs
                rel = np.expm1(dz) + n * 2.0 ** -24
                if form == "decode":
                    tol = 2 * vmax * (rel + 2.0 ** -20) + 1e-37
                else:
                    tol = np.abs(o) * 2.0 ** -8 + 2 * vmax * (rel + 2.0 ** -11 + n * 2.0 ** -31) + 2.0 ** -133
                    if pool.kind in ("bf16", "fp8k"):
                        tol = tol + 2.0 ** -17
                err = np.abs(got[row, h] - o)
                assert (err <= tol).all(), (s, L, P, h, float((err / tol).max()), float(err.max()))
            row += 1


LENS = np.array([0, 1, 15, 16, 17, 100, 128, 129, 300])


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,bs,Hq,H,W,S", [(64, 16, 4, 2, 0, 4), (128, 16, 8, 2, 5, 1), (128, 32, 24, 2, 100, 17),
                                           (256, 16, 3, 1, 16, 16), (128, 64, 7, 7, 33, 200), (64, 16, 16, 1, 1, 0),
                                           (128, 256, 10, 2, 64, 40)])
def test_decode_with_sinks(kind, split, D, bs, Hq, H, W, S):
    rng = np.random.default_rng(W * 31 + S + D)
    new = np.ones(len(LENS), np.int64)
    pool = Pool(rng, kind, LENS, new, H, D, bs, W, S)
    q = bf16(rng.standard_normal((len(LENS), Hq * D + 8))).to(DEV)
    out = torch.full((len(LENS), Hq, D), float("nan"), device=DEV)
    ws = torch.empty(pk.kv_decode_workspace_bytes(pool.tables.shape[1], len(LENS), Hq, H, D, bs), dtype=torch.uint8,
                     device=DEV) if split else None
    pk.kv_set_decode_workspace(ws)
    call(pool, "decode", q, out, LENS, None, Hq, W, S, q_stride=Hq * D + 8)
    check_rows(pool, "decode", q, out, LENS, new, Hq, W, S)
    assert pk.kv_get_device_error() == 0
    pk.kv_set_decode_workspace(None)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_sums_of_a_long_sequence(kind):
    """30,000 positions in one sum (no workspace), V positive so that nothing cancels. 1,875 tiles are added to nearest,
    each addition off by at most 2^-24 of a sum that grows evenly: a third of their squares on average, so 6 sigma is 6
    sqrt(1875 / 3) 2^-24 = 9e-6 of the result. Scores: dz = (D + 8) 2^-23 |z| at most, of alternating sign over the
    positions; with the weights' 2^-22 another 2^-19 covers them. (Additions towards zero would be 1,875 times half of
    2^-23 times a half: 5.6e-5.)"""
    rng = np.random.default_rng(17)
    L, D, H, bs = 30000, 64, 1, 256
    pool = Pool(rng, kind, [L], [1], H, D, bs, 0, 0)
    v = pool.raw[1]
    pool.raw[1] = v & 0x7F if v.dtype == torch.uint8 else v.abs()
    if pool.scales:
        pool.scales[1][:] = 2.0 ** -5                     # one scale, so that every position weighs alike
        pool.rows[1][0] = ref.e4m3_values(pool.raw[1].cpu().numpy())[pool.tables[0, np.arange(L) // bs],
                                                                    np.arange(L) % bs] * 2.0 ** -5
    q = bf16(rng.standard_normal((1, 2 * D))).to(DEV)
    out = torch.full((1, 2, D), float("nan"), device=DEV)
    pk.kv_set_decode_workspace(None)
    call(pool, "decode", q, out, [L], None, 2, 0, 0)
    want = np.stack([ref.attention(f64(q).reshape(2, D)[h], pool.rows[0][0][:, 0], np.abs(pool.rows[1][0][:, 0]), L - 1, 0,
                                   0, D ** -0.5)[0] for h in range(2)])
    err = np.linalg.norm(f64(out)[0] - want) / np.linalg.norm(want)
    assert err <= 9e-6 + 2.0 ** -19, err


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,bs,Hq,H,W,S", [(64, 16, 4, 2, 0, 4), (128, 16, 8, 2, 5, 1), (128, 32, 6, 2, 100, 17),
                                           (128, 64, 3, 3, 33, 200), (64, 16, 16, 1, 1, 0), (64, 128, 5, 1, 20, 129),
                                           (128, 16, 4, 1, 130, 64)])
def test_prefill_with_sinks(kind, D, bs, Hq, H, W, S):
    rng = np.random.default_rng(W * 37 + S + D)
    lens = np.array([1, 17, 0, 129, 300, 40, 700, 33])
    new = np.array([1, 17, 0, 70, 9, 0, 3, 33])
    pool = Pool(rng, kind, lens, new, H, D, bs, W, S)
    T = int(new.sum())
    q = bf16(rng.standard_normal((T + 3, Hq * D))).to(DEV)
    out = torch.full((T + 3, Hq, D), 7.0, device=DEV, dtype=torch.bfloat16)
    call(pool, "prefill", q, out, lens, np.concatenate([[0], np.cumsum(new)]), Hq, W, S)
    check_rows(pool, "prefill", q[:T], out[:T], lens, new, Hq, W, S)
    assert bool((out[T:] == 7.0).all()), "rows behind the last sequence were written"
    assert pk.kv_get_device_error() == 0


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_block_scales_of_any_size(form):
    """V scales from 2^-24 to 2^24 from block to block, some not powers of two: each row's error stays small against
    the values that it attends."""
    rng = np.random.default_rng(8)
    lens, new = np.array([200, 64, 1000]), np.array([1, 1, 1]) if form == "decode" else np.array([40, 64, 5])
    pool = Pool(rng, "fp8_block", lens, new, 2, 128, 16, 0, 0, wide=True)
    T = int(new.sum())
    q = bf16(rng.standard_normal((T, 4 * 128)) * 3).to(DEV)
    out = torch.empty((T, 4, 128), device=DEV, dtype=torch.float32 if form == "decode" else torch.bfloat16)
    call(pool, form, q, out, lens, np.concatenate([[0], np.cumsum(new)]), 4, 0, 0)
    check_rows(pool, form, q, out, lens, new, 4, 0, 0)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("kind", KINDS)
def test_queries_near_the_smallest_numbers(kind, form):
    """Queries of 2^-120 (and least K scales): every score is 0 but for 2^-100, the masked ones among them."""
    rng = np.random.default_rng(12)
    lens, new = np.array([200, 64, 300]), np.array([1, 1, 1]) if form == "decode" else np.array([40, 64, 5])
    pool = Pool(rng, kind, lens, new, 2, 128, 16, 30, 4)
    if pool.scales:
        live = np.isfinite(pool.scales[0])
        for s, L in enumerate(lens):                      # the reference's keys at the new scale
            blk = pool.tables[s, np.arange(L) // 16]
            old = np.where(live[blk], pool.scales[0][blk], 1.0).astype(np.float64)
            pool.rows[0][s] = pool.rows[0][s] / old[..., None] * 2.0 ** -60
        pool.scales[0][live] = 2.0 ** -60
    T = int(new.sum())
    q = bf16(rng.standard_normal((T, 4 * 128)) * 2.0 ** -120).to(DEV)
    out = torch.empty((T, 4, 128), device=DEV, dtype=torch.float32 if form == "decode" else torch.bfloat16)
    call(pool, form, q, out, lens, np.concatenate([[0], np.cumsum(new)]), 4, 30, 4)
    check_rows(pool, form, q, out, lens, new, 4, 30, 4)


@pytest.mark.parametrize("kind", KINDS)
def test_queries_before_the_first_position_give_zeros(kind):
    rng = np.random.default_rng(3)
    lens, new = np.array([4, 0]), np.array([9, 3])           # more queries than positions
    pool = Pool(rng, kind, lens, np.array([4, 0]), 1, 128, 16, 0, 0)
    q = bf16(rng.standard_normal((12, 256))).to(DEV)
    out = torch.full((12, 2, 128), float("nan"), device=DEV, dtype=torch.bfloat16)
    call(pool, "prefill", q, out, lens, [0, 9, 12], 2, 2, 1)
    check_rows(pool, "prefill", q, out, lens, new, 2, 2, 1)
    assert bool((out[:5] == 0).all()) and bool((out[9:] == 0).all())


@pytest.mark.parametrize("kind", KINDS)
def test_sinks_change_nothing_without_a_window(kind):
    """num_sinks without a window, and a window with no sinks, give the plain calls' values. The prefill's bits where
    there is no window (BF16 rows: their rounding); with one it begins its key tiles elsewhere, so that both are within
    the weights' rounding of the same value (2 max|v| 2^-11 each, and the sums' 2^-18), `out` rounded to BF16 besides.
    The decode adds its tiles to nearest, the plain one towards zero: 2 products for each of 19 tiles, each cut by at most
    2^-23 of a sum that is on average half of max|v| times the weights' sum, 2^-18.75 in all. The weights have 22 bits over
    an E4M3 V (each side 2 max|v| 2^-22), over a BF16 V the plain call's have 16 (2 max|v| 2^-17)."""
    rng = np.random.default_rng(4)
    lens, new = np.array([300, 17]), np.array([50, 17])
    pool = Pool(rng, kind, lens, new, 2, 128, 16, 0, 0)
    q = bf16(rng.standard_normal((67, 512))).to(DEV)
    outs = []
    for S in (0, 5):
        out = torch.empty((67, 4, 128), device=DEV, dtype=torch.bfloat16)
        call(pool, "prefill", q, out, lens, [0, 50, 67], 4, 0, S)
        dec = torch.empty((2, 4, 128), device=DEV)
        call(pool, "decode", q[:2], dec, lens, None, 4, 0, S)
        outs.append((out, dec))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    if kind == "fp8_block":
        return
    tail = [pool.tables.shape[1], 2]
    for W in (0, 40):
        pre, dec = torch.empty((67, 4, 128), device=DEV), torch.empty((2, 4, 128), device=DEV)
        getattr(pk, f"paged_prefill_attn_{kind}")(q, *pool.raw, pre, i32(pool.tables), i32(lens), i32([0, 50, 67]), *tail,
                                                  67, 4, 2, 128, 16, 128 ** -0.5, *pool.scalars(), 512, W)
        getattr(pk, f"paged_decode_attn_{kind}")(q[:2].contiguous(), *pool.raw, dec, i32(pool.tables), i32(lens), *tail, 4,
                                                 2, 128, 16, 128 ** -0.5, *pool.scalars(), 512, W)
        out = torch.empty((67, 4, 128), device=DEV, dtype=torch.bfloat16)
        call(pool, "prefill", q, out, lens, [0, 50, 67], 4, W, 0)
        one = torch.empty((2, 4, 128), device=DEV)
        call(pool, "decode", q[:2], one, lens, None, 4, W, 0)
        vmax = max(np.abs(v).max() for v in pool.rows[1])
        weights = 2 * 2.0 ** -22 if kind == "fp8" else 2.0 ** -17
        assert float((dec - one).abs().max()) <= 2 * vmax * (weights + 2.0 ** -18)
        if W == 0:
            assert torch.equal(pre.to(torch.bfloat16), out)
        else:
            tol = 4 * vmax * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -8 * pre.abs() + 2.0 ** -16
            assert bool(((pre - out.float()).abs() <= tol).all())


def test_calls_in_a_captured_graph():
    """Write and decode captured once, replayed with other tokens, lengths and query rows."""
    rng = np.random.default_rng(21)
    H, Hq, D, bs, B = 2, 8, 128, 16, 3
    lens = np.array([30, 1, 64])
    tables, nb = permuted_tables(rng, lens + 40, bs)
    cache = Cache(nb, bs, H, D)
    qsl = np.arange(B + 1)
    width = tables.shape[1]
    d_tables, d_lens, d_qsl = i32(tables), i32(lens), i32(qsl)
    key, value = torch.zeros((B, H * D), device=DEV, dtype=torch.bfloat16), torch.zeros((B, H * D), device=DEV,
                                                                                       dtype=torch.bfloat16)
    q, out = torch.zeros((B, Hq * D), device=DEV, dtype=torch.bfloat16), torch.empty((B, Hq, D), device=DEV)
    # the earlier tokens
    T = int(lens.sum()) - B
    prompt = [bf16(rng.standard_normal((T, H * D))) for _ in range(2)]
    write_both(cache, *prompt, tables, lens - 1, np.concatenate([[0], np.cumsum(lens - 1)]), H, D, bs)
    ws = torch.empty(pk.kv_decode_workspace_bytes(width, B, Hq, H, D, bs), dtype=torch.uint8, device=DEV)
    pk.kv_set_decode_workspace(ws)

    def step():
        pk.kv_write_fp8_block(key, value, *cache.dc, *cache.ds, d_tables, d_lens, d_qsl, width, B, B, H, D, bs, H * D,
                              H * D)
        pk.paged_decode_attn_fp8_block(q, *cache.dc, *cache.ds, out, d_tables, d_lens, width, B, Hq, H, D, bs,
                                       D ** -0.5, Hq * D, 20, 3)
    fill = lambda t: t.copy_(bf16(rng.standard_normal(t.shape)))  # noqa: E731
    for t in (key, value, q):
        fill(t)
    step()
    ref.write_block(f64(key), f64(value), cache.codes, cache.scales, tables, lens, qsl, H, D, bs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for t in (key, value, q):
            fill(t)
        d_lens += 1
        lens = lens + 1
        graph.replay()
        ref.write_block(f64(key), f64(value), cache.codes, cache.scales, tables, lens, qsl, H, D, bs)
        cache.check()
        want = torch.empty_like(out)
        pk.kv_set_decode_workspace(None)
        pk.paged_decode_attn_fp8_block(q, *cache.dc, *cache.ds, want, d_tables, d_lens, width, B, Hq, H, D, bs,
                                       D ** -0.5, Hq * D, 20, 3)
        pk.kv_set_decode_workspace(ws)
        assert torch.allclose(out, want, atol=1e-5, rtol=0)  # split and unsplit sums: a few 2^-20 of max|v| < 5
    pk.kv_set_decode_workspace(None)
