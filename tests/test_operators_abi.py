"""Argument checks of the block-scaled cache, the calls with sinks and the page
calls, before any CUDA call is made, and the references that the GPU tests
compare with (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import reference64 as ref

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)
BAD = (0.0, -1.0, float("inf"), float("nan"))


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_fill_gb300 import _build
    _build.build()
    import paged_kv_cache_fill_gb300 as pk
    pk.lib()
    return pk


def write(L, **kw):
    a = dict(key=FAKE, value=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, mbps=4, ns=2, nt=3,
             H=8, D=128, bs=16, kst=1024, vst=1024)
    a.update(kw)
    return L.kv_write_fp8_block(*a.values(), None)


def attn(L, form, kind, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, out=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, mbps=4, ns=2, nq=10, Hq=32,
             H=8, D=128, bs=16, isd=0.1, k_scale=1.0, v_scale=1.0, q_stride=4096, win=64, sinks=4)
    a.update(kw)
    if kind != "fp8_block":
        del a["ks"], a["vs"]
    if kind != "fp8":
        del a["v_scale"]
    if kind not in ("fp8", "fp8k"):
        del a["k_scale"]
    if form == "decode":
        del a["qsl"], a["nq"]
    name = f"paged_{form}_attn_{kind}" + ("" if kind == "fp8_block" else "_sinks")
    return getattr(L, name)(*a.values(), None)


KINDS = ["bf16", "fp8k", "fp8", "fp8_block"]


def test_write_block_refusals(pk):
    L, INV, UNS = pk.lib(), pk.KV_ERR_INVALID_ARG, pk.KV_ERR_UNSUPPORTED
    none = dict.fromkeys(["key", "value", "kc", "vc", "ks", "vs", "bt", "sl", "qsl"])
    assert write(L, nt=0, **none) == pk.KV_OK and write(L, ns=0, **none) == pk.KV_OK
    for name in none:
        assert write(L, **{name: None}) == INV, name
    assert write(L, H=0) == INV and write(L, D=0) == INV and write(L, bs=0) == INV
    assert write(L, kst=1023) == INV and write(L, vst=1000) == INV
    assert write(L, D=96) == UNS and write(L, D=512, kst=4096, vst=4096) == UNS
    assert write(L, bs=8) == UNS and write(L, bs=24) == UNS and write(L, bs=512) == UNS
    assert write(L, kc=ODD) == UNS and write(L, vc=ODD) == UNS
    assert write(L, mbps=1 << 27) == UNS and write(L, nt=1 << 31) == UNS


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_attention_refusals(pk, form, kind):
    L, INV, UNS = pk.lib(), pk.KV_ERR_INVALID_ARG, pk.KV_ERR_UNSUPPORTED
    none = dict(q=None, k=None, v=None, out=None)
    assert attn(L, form, kind, ns=0, **none) == pk.KV_OK
    for name in ("q", "k", "v", "out", "bt", "sl"):
        assert attn(L, form, kind, **{name: None}) == INV, name
    assert attn(L, form, kind, Hq=30) == INV and attn(L, form, kind, H=0) == INV
    assert attn(L, form, kind, q_stride=100) == INV and attn(L, form, kind, isd=float("nan")) == INV
    assert attn(L, form, kind, D=96, q_stride=32 * 96) == UNS
    assert attn(L, form, kind, bs=8) == UNS and attn(L, form, kind, bs=24) == UNS
    assert attn(L, form, kind, q=ODD) == UNS and attn(L, form, kind, v=ODD) == UNS
    assert attn(L, form, kind, q_stride=4100) == UNS and attn(L, form, kind, mbps=1 << 27) == UNS
    if kind == "fp8_block":
        assert attn(L, form, kind, ks=None) == INV and attn(L, form, kind, vs=None) == INV
    if kind in ("fp8k", "fp8"):
        assert all(attn(L, form, kind, k_scale=x) == INV for x in BAD)
    if kind == "fp8":
        assert all(attn(L, form, kind, v_scale=x) == INV for x in BAD)
    if form == "prefill":
        assert attn(L, form, kind, nq=0, **none) == pk.KV_OK and attn(L, form, kind, qsl=None) == INV
        assert all(attn(L, form, kind, isd=x) == INV for x in BAD)
        assert attn(L, form, kind, D=256, q_stride=32 * 256) == UNS and attn(L, form, kind, out=ODD) == UNS
    else:
        assert attn(L, form, kind, Hq=256, q_stride=256 * 128) == UNS      # 32 query heads per KV head


def test_page_call_refusals(pk):
    L, INV, UNS, OK = pk.lib(), pk.KV_ERR_INVALID_ARG, pk.KV_ERR_UNSUPPORTED, pk.KV_OK
    bases, sizes = (ctypes.c_void_p * 2)(0x10000, 0x20000), (ctypes.c_size_t * 2)(64, 64)
    copy = lambda p=bases, b=sizes, n=2, s=FAKE, d=FAKE, k=3, nb=9: L.kv_copy_blocks(p, b, n, s, d, k, nb, None)  # noqa: E731
    assert copy(None, None, 0) == OK and copy(None, None, s=None, d=None, k=0) == OK
    assert copy(p=None) == INV and copy(b=None) == INV and copy(s=None) == INV and copy(d=None) == INV
    assert copy(nb=0) == INV and copy(p=(ctypes.c_void_p * 2)(0x10000, None)) == INV
    assert copy(b=(ctypes.c_size_t * 2)(64, 0)) == INV and copy(b=(ctypes.c_size_t * 2)(64, 1 << 40)) == UNS
    assert copy(nb=1 << 31) == UNS and copy(k=1 << 31) == UNS
    free = lambda t=FAKE, r=FAKE, f=FAKE, e=FAKE, w=4, s=2, nb=9: L.kv_free_blocks(t, r, f, e, w, s, nb, None)  # noqa: E731
    assert free(None, None, None, None, s=0) == OK
    assert free(t=None) == INV and free(r=None) == INV and free(f=None) == INV and free(e=None) == INV
    assert free(w=0) == INV and free(nb=0) == INV and free(nb=1 << 31) == UNS
    win = lambda t=FAKE, r=FAKE, n=FAKE, w=4, s=2, nb=9, bs=16, W=5: L.kv_free_window_blocks(  # noqa: E731
        t, r, n, w, s, nb, bs, W, 1, None)
    assert win(None, None, None, s=0) == OK and win(None, None, None, W=0) == OK
    assert win(t=None) == INV and win(r=None) == INV and win(n=None) == INV and win(bs=0) == INV and win(nb=0) == INV

    def fork(n=1, w=4, s=3, nb=9, bs=16, **kw):
        a = dict.fromkeys(["t", "sl", "r", "src", "dst", "cs", "cd"], FAKE)
        a.update(kw)
        return L.kv_fork_blocks(*a.values(), n, w, s, nb, bs, None)
    assert fork(n=0, t=None) == OK
    assert all(fork(**{x: None}) == INV for x in ("t", "sl", "r", "src", "dst", "cs", "cd"))
    assert fork(s=0) == INV and fork(bs=0) == INV and fork(w=0) == INV and fork(nb=0) == INV
    assert fork(r=ODD) == UNS and fork(nb=1 << 31) == UNS and fork(n=60000) == UNS and fork(s=1 << 20) == UNS

    def compact(w=4, s=3, nb=9, **kw):
        a = dict.fromkeys(["t", "r", "nt", "nr", "ids", "cs", "cd", "u"], FAKE)
        a.update(kw)
        return L.kv_compact_blocks(*a.values(), w, s, nb, None)
    assert compact(nb=0, t=None) == OK
    assert all(compact(**{x: None}) == INV for x in ("t", "r", "nt", "nr", "ids", "cs", "cd", "u"))
    assert compact(w=0) == INV and compact(nb=1 << 31) == UNS


def test_binding_refuses_host_tensors(pk):
    t = torch.zeros(4, dtype=torch.int32)
    if torch.cuda.is_available():
        pytest.skip("the binding's checks on a GPU host are tested there")
    for call in (lambda: pk.kv_copy_blocks([t], t, t, 1, 4), lambda: pk.kv_free_blocks(t, t, t, t, 1, 1, 4),
                 lambda: pk.kv_fork_blocks(t, t, t, t, t, t, t, 1, 1, 4, 4, 16)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


# ---------------------------------------------------------------------------
# the references themselves
# ---------------------------------------------------------------------------
def test_reference_e4m3_is_the_format():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.e4m3_values(codes), want, equal_nan=True)
    finite = codes[~np.isnan(want)]
    assert np.array_equal(ref.e4m3_codes(ref.e4m3_values(finite)), finite)
    # halfway cases go to the even code, values past the largest saturate
    v = ref.e4m3_values(np.arange(0, 127, dtype=np.uint8))
    mid = (v[:-1] + v[1:]) / 2
    assert np.array_equal(ref.e4m3_codes(mid), np.arange(0, 126) + np.arange(0, 126) % 2)
    assert ref.e4m3_codes(np.array([1e9, -1e9, np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7E, 0x7F]


def test_copy_refuses_one_tensor_as_the_pools(pk):
    """Taken as a sequence, a pool would be copied as num_blocks pools of a block each."""
    ids = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="sequence"):
        pk.kv_copy_blocks(torch.zeros(4, 4, 64, dtype=torch.uint8), ids, ids, 1, 4)


def test_reference_scale_is_least():
    for amax in (448.0, 448.0001, 1.0, 3e38, 2.0 ** -60, 0.0, 1.75 * 2.0 ** -40, 1.7500001 * 2.0 ** -40):
        s = ref.pow2_scale(amax)
        assert amax <= 448 * s and (s == 2.0 ** -60 or amax > 448 * s / 2)
    assert ref.pow2_scale(0.0) == 2.0 ** -60


def test_reference_attended_positions():
    assert ref.attended(9, 0, 3).tolist() == list(range(10))
    assert ref.attended(9, 4, 2).tolist() == [0, 1, 6, 7, 8, 9]
    assert ref.attended(2, 4, 2).tolist() == [0, 1, 2]
    assert ref.attended(9, 4, 99).tolist() == list(range(10))


def test_reference_fork_and_compact_keep_every_page():
    """A fork's row reads what its parent's did, and compaction moves each block's content to its new id."""
    rng = np.random.default_rng(3)
    bs, nb = 16, 40
    tables = np.full((4, 5), -1, np.int32)
    refs = np.zeros(nb, np.int32)
    perm = rng.permutation(nb)
    lens = np.array([70, 32, 0, 0], np.int32)
    tables[0], tables[1, :2] = perm[:5], perm[5:7]
    refs[perm[:7]] = 1
    data = rng.integers(0, 1000, nb)
    s, d = ref.fork_blocks(tables, lens, refs, [0, 1], [2, 3], bs)
    data[d[s >= 0]] = data[s[s >= 0]]
    assert np.array_equal(data[tables[0]], data[tables[2]]) and tables[2, 4] != tables[0, 4]
    assert np.array_equal(tables[1], tables[3]) and s.tolist()[1] == -1
    assert all(refs[b] == (tables == b).sum() for b in range(nb))
    t, r, ids, cs, cd, used = ref.compact_blocks(tables, refs)
    moved = data.copy()
    moved[cd[cd >= 0]] = data[cs[cs >= 0]]
    live = tables >= 0
    assert np.array_equal(moved[t[live]], data[tables[live]]) and t.max() == used - 1
    assert all(r[b] == (t == b).sum() for b in range(nb))
