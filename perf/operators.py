"""Cases of the block-scaled FP8 cache, of attention with sinks and of page moves.

Five operators of a paged KV-cache server, each over the range of sizes that
such a server meets:

  write    kv_write_fp8_block: keys and values into an E4M3 cache with one
           power-of-two scale for each (block of tokens, KV head).
  decode   one query token per sequence over a paged cache, with a sliding
           window and first tokens that stay visible (sinks):
           paged_decode_attn_fp8_block and the `_sinks` calls of the BF16,
           FP8-K and FP8 caches.
  prefill  the same for chunks of query tokens (paged_prefill_attn_*).
  fork     kv_free_blocks, kv_fork_blocks and kv_copy_blocks: the children of
           the last step let go of their pages and become forks of their
           parents, sharing full pages and copying the partial one.
  compact  kv_compact_blocks and kv_copy_blocks: the used pages of a
           fragmented pool move to the lowest ids.

Where `own` is false, run() computes them from elementary torch operations in
32 bits; where it is true it makes the library's calls. exact() computes the
floating-point ones in 64 bits, sequence by sequence.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -60  # the write's smallest block scale
NAN_CODE = 0x7F

_ws = None  # the library's split-KV workspace, registered once and kept


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a small server appends one token per sequence
        dict(name="write-append-64", op="write", seqs=64, min_len=512, max_len=8192, min_new=1, max_new=1,
             empty=0, heads=8, dim=128, block=16, pad=0),
        # chunks of prompts, ragged, keys and values taken out of a fused projection's rows
        dict(name="write-prompts-24", op="write", seqs=24, min_len=4097, max_len=9001, min_new=3001,
             max_new=7923, empty=0, heads=8, dim=128, block=64, pad=2048),
        # one interactive user: latency
        dict(name="decode-block-2", op="decode", kind="fp8_block", seqs=2, min_len=37, max_len=100, empty=0, heads=2,
             group=2, dim=64, block=16, window=0, sinks=0),
        # long documents, whole context
        dict(name="decode-block-64x32768", op="decode", kind="fp8_block", seqs=64, min_len=32768, max_len=32768,
             empty=0, heads=8, group=4, dim=128, block=16, window=0, sinks=0),
        # streaming dialogues: long past, a window and four sinks, pages in between given back
        dict(name="decode-bf16-sinks-64", op="decode", kind="bf16", seqs=64, min_len=512, max_len=8192, empty=1,
             heads=8, group=4, dim=128, block=16, window=1000, sinks=4),
        # prompts of a tiny model, odd lengths: latency
        dict(name="prefill-block-2", op="prefill", kind="fp8_block", seqs=2, min_len=37, max_len=100, min_new=20,
             max_new=37, empty=0, heads=2, group=2, dim=64, block=16, window=0, sinks=0),
        # chunked prefill of documents
        dict(name="prefill-block-8x1024", op="prefill", kind="fp8_block", seqs=8, min_len=4096, max_len=8192,
             min_new=1024, max_new=1024, empty=0, heads=8, group=4, dim=128, block=16, window=0, sinks=0),
        # chunked prefill with a window and sinks, ragged
        dict(name="prefill-bf16-sinks-16", op="prefill", kind="bf16", seqs=16, min_len=1500, max_len=16384,
             min_new=200, max_new=1500, empty=1, heads=8, group=4, dim=128, block=16, window=1024, sinks=4),
        # beam search over a few prompts
        dict(name="fork-beams-8x4", op="fork", parents=8, children=3, min_len=100, max_len=1000, layers=4, heads=8,
             dim=128, block=16, blocks=2048),
        # many samples from each prompt of a large model: every partial page of every layer is copied
        dict(name="fork-samples-32x15", op="fork", parents=32, children=15, min_len=500, max_len=4000, layers=32,
             heads=8, dim=128, block=64, blocks=4096),
        # a small pool after a few requests have finished
        dict(name="compact-512", op="compact", blocks=512, used=0.4, max_blocks=64, layers=2, heads=8, dim=128,
             block=16),
        # a large pool after hours of serving
        dict(name="compact-16384", op="compact", blocks=16384, used=0.55, max_blocks=512, layers=8, heads=8, dim=128,
             block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prefill", "prefill", "fork", "compact"])
    block = rng.choice([16, 16, 32, 64, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 128])
    if op == "write":
        dim = rng.choice([64, 128, 256])
        seqs = _log(rng, 1, 200)
        top = max(2, min(8000, 100000 // seqs))
        new = _log(rng, 1, top)
        lo = _log(rng, new, new + 4000)
        return dict(op=op, seqs=seqs, min_len=lo, max_len=lo + _log(rng, 1, 3000), min_new=max(1, new // 2),
                    max_new=new, empty=rng.choice([0, 0, 1, 3]), heads=heads, dim=dim, block=block,
                    pad=rng.choice([0, 8, 256, 3]))
    if op == "decode":
        kind = rng.choice(["fp8_block", "fp8_block", "bf16", "fp8k", "fp8"])
        dim = rng.choice([64, 128, 128, 256]) if kind != "fp8" else rng.choice([128, 128, 256])
        seqs = _log(rng, 1, 200)
        hi = _log(rng, 1, max(2, min(40000, 1500000 // seqs)))
        window = rng.choice([0, _log(rng, 1, 4096), _log(rng, 64, 4096)])
        return dict(op=op, kind=kind, seqs=seqs, min_len=max(1, hi // rng.choice([1, 3, 20])), max_len=hi,
                    empty=rng.choice([0, 0, 1, 2]), heads=heads, group=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]),
                    dim=dim, block=block, window=window, sinks=rng.choice([0, 1, 4, 16, 17, 100]))
    if op == "prefill":
        kind = rng.choice(["fp8_block", "fp8_block", "bf16", "fp8k", "fp8"])
        seqs = _log(rng, 1, 24)
        new = _log(rng, 1, max(2, 4096 // seqs))
        past = _log(rng, 1, max(2, min(16000, 40000 // seqs)))
        window = rng.choice([0, _log(rng, 1, 2048), _log(rng, 64, 2048)])
        return dict(op=op, kind=kind, seqs=seqs, min_len=new + past // 3, max_len=new + past,
                    min_new=max(1, new // 3), max_new=new, empty=rng.choice([0, 0, 1, 2]), heads=heads,
                    group=rng.choice([1, 2, 3, 4, 5, 7, 8]), dim=dim, block=block, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 17, 100, 200]))
    if op == "fork":
        parents, children = _log(rng, 1, 32), _log(rng, 1, 15)
        lo = _log(rng, 1, 1000)
        hi = lo + _log(rng, 1, 2000)
        need = parents * (-(-hi // block) + children + 1)
        return dict(op=op, parents=parents, children=children, min_len=lo, max_len=hi, layers=_log(rng, 1, 8),
                    heads=heads, dim=dim, block=block, blocks=need + _log(rng, 1, 2 * need))
    return dict(op=op, blocks=_log(rng, 50, 8000), used=rng.uniform(0.05, 0.95), max_blocks=_log(rng, 8, 300),
                layers=_log(rng, 1, 4), heads=heads, dim=dim, block=min(block, 64))


def _attended(case, L, n=1):
    """Key positions that the last n queries of a sequence of length L attend, as (first of them that are sinks, first
    of the rest)."""
    W, S = case["window"], case["sinks"]
    lo = max(0, L - n + 1 - W) if W else 0
    return min(S, lo), lo


def _lens(case):
    """The sequences' lengths and new tokens: spread evenly over the case's range on a logarithmic scale, in an order
    that does not sort them; the last `empty` sequences are empty."""
    B = case["seqs"]
    empty = min(case.get("empty", 0), B - 1)
    lo, hi = case["min_len"], case["max_len"]
    lens = [int(round(math.exp(math.log(lo) + ((i * 7 + 3) % B + 0.5) / B * (math.log(hi) - math.log(lo)))))
            for i in range(B)]
    new = [1] * B
    if "max_new" in case:
        a, b = case["min_new"], case["max_new"]
        new = [min(lens[i], a + (b - a) * ((i * 5 + 2) % B) // max(1, B - 1)) for i in range(B)]
    for i in range(B - empty, B):
        lens[i], new[i] = 0, 0
    return lens, new


def _parents(case):
    P, lo, hi = case["parents"], case["min_len"], case["max_len"]
    return [lo + (hi - lo) * ((i * 3 + 1) % P) // max(1, P - 1) for i in range(P)]


def _used(case):
    return max(1, min(case["blocks"] - 1, int(case["blocks"] * case["used"])))


def work(case):
    op = case["op"]
    H, D = case["heads"], case["dim"]
    if op == "write":
        lens, new = _lens(case)
        T, bs = sum(new), case["block"]
        touched = sum((L - 1) // bs - (L - n) // bs + 1 for L, n in zip(lens, new) if n)
        return {"bytes": T * H * D * 6 + touched * (H * 16 + 4), "flops": T * H * D * 4}
    if op in ("decode", "prefill"):
        lens, new = _lens(case)
        Hq = H * case["group"]
        kb = {"bf16": 2, "fp8k": 1, "fp8": 1, "fp8_block": 1}[case["kind"]]
        vb = {"bf16": 2, "fp8k": 2, "fp8": 1, "fp8_block": 1}[case["kind"]]
        sb = 8 / case["block"] if case["kind"] == "fp8_block" else 0
        rows = pairs = 0
        for L, n in zip(lens, new):
            s, lo = _attended(case, L, n)
            rows += s + L - lo if n else 0
            for P in {L - 1} if n == 1 else range(L - n, L):
                s, lo = _attended(case, P + 1)
                pairs += s + P + 1 - lo if n else 0
        T = sum(new) if op == "prefill" else len(lens)
        ob = 2 if op == "prefill" else 4
        return {"bytes": rows * H * (D * (kb + vb) + sb) + T * Hq * D * (2 + ob), "flops": pairs * Hq * D * 4}
    page = case["block"] * H * D * 2 + H * 8  # K and V codes and their scales, one layer
    if op == "fork":
        bs = case["block"]
        part = sum(1 for L in _parents(case) if L % bs)
        rows = sum(-(-L // bs) for L in _parents(case))
        return {"bytes": case["children"] * (2 * part * case["layers"] * page + 3 * 4 * rows), "flops": 0}
    U, N = _used(case), case["blocks"]
    moved = U * (N - U) // N
    return {"bytes": 2 * moved * case["layers"] * page + 12 * N + 8 * U, "flops": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least MIN_SCALE (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp_min(MIN_SCALE)


def _block_pool(g, nb, bs, H, D, sigma):
    """An E4M3 pool and its scales: N(0, sigma_h) with a spread of magnitudes from block to block."""
    codes = torch.empty((nb, bs, H, D), dtype=torch.uint8, device=DEV)
    scales = torch.empty((nb, H), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (bs * H * D))
    for b in range(0, nb, step):
        n = min(step, nb - b)
        x = torch.randn((n, bs, H, D), generator=g, device=DEV)
        x *= sigma[None, None, :, None] * torch.exp(0.3 * torch.randn((n, 1, H, 1), generator=g, device=DEV))
        s = _pow2_scale(x.abs().amax((1, 3)))
        scales[b:b + n] = s
        codes[b:b + n] = (x / s[:, None, :, None]).to(E4M3).view(torch.uint8)
    return codes, scales


def _pool(g, nb, bs, H, D, dtype):
    out = torch.empty((nb, bs, H, D), dtype=dtype, device=DEV)
    step = max(1, (1 << 27) // (bs * H * D))
    for b in range(0, nb, step):
        x = torch.randn((min(step, nb - b), bs, H, D), generator=g, device=DEV)
        out[b:b + step] = x.to(dtype) if dtype != torch.uint8 else (x * 60).clamp(-448, 448).to(E4M3).view(dtype)
    return out


def _tables(g, lens, bs, nb, width):
    """Block tables over a shuffled pool; entries past a sequence's blocks are -1."""
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).cpu()
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, L in enumerate(lens):
        n = -(-L // bs)
        t[s, :n] = perm[at:at + n]
        at += n
    return t.to(DEV), perm[at:].to(DEV).long()


def prepare(case, seed):
    g = _gen(seed)
    return {"write": _prepare_write, "decode": _prepare_attn, "prefill": _prepare_attn, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, g)


def _prepare_write(case, g):
    H, D, bs = case["heads"], case["dim"], case["block"]
    lens, new = _lens(case)
    width = max(1, max(-(-L // bs) for L in lens))
    nb = sum(-(-L // bs) for L in lens) + 5
    tables, _ = _tables(g, lens, bs, nb, width)
    T, row = sum(new), H * D
    stride = row + case["pad"]
    sigma = torch.tensor([1.0, 4.0, 18.0], device=DEV)[torch.randint(0, 3, (H,), generator=g, device=DEV)]
    key = torch.randn((T, stride), generator=g, device=DEV)
    key[:, :row] *= sigma.repeat_interleave(D)
    value = torch.randn((T, stride), generator=g, device=DEV)
    kc, ks = _block_pool(g, nb, bs, H, D, 0.5 * sigma)
    vc, vs = _block_pool(g, nb, bs, H, D, torch.ones(H, device=DEV))
    qsl = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    return dict(op="write", case=case, key=key.to(torch.bfloat16), value=value.to(torch.bfloat16), kc=kc, vc=vc,
                ks=ks, vs=vs, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), qsl=qsl,
                width=width, tokens=T, stride=stride)


def _prepare_attn(case, g):
    H, G, D, bs = case["heads"], case["group"], case["dim"], case["block"]
    lens, new = _lens(case)
    width = max(1, max(-(-L // bs) for L in lens))
    nb = sum(-(-L // bs) for L in lens) + 5
    tables, spare = _tables(g, lens, bs, nb, width)
    kind = case["kind"]
    st = dict(op=case["op"], case=case, ks=None, vs=None)
    if kind == "fp8_block":
        sigma = torch.tensor([0.5, 1.0, 2.0], device=DEV)[torch.randint(0, 3, (H,), generator=g, device=DEV)]
        st["kc"], st["ks"] = _block_pool(g, nb, bs, H, D, sigma)
        st["vc"], st["vs"] = _block_pool(g, nb, bs, H, D, torch.ones(H, device=DEV))
    else:
        st["kc"] = _pool(g, nb, bs, H, D, torch.bfloat16 if kind == "bf16" else torch.uint8)
        st["vc"] = _pool(g, nb, bs, H, D, torch.uint8 if kind == "fp8" else torch.bfloat16)
    # rows past a sequence's end and pages that no table names hold NaN
    for c in (st["kc"], st["vc"]):
        nan = NAN_CODE if c.dtype == torch.uint8 else math.nan
        c[spare] = nan
        for s, L in enumerate(lens):
            if L % bs:
                c[tables[s, L // bs].long(), L % bs:] = nan
    # pages that no query attends any more have been given back
    for s, (L, n) in enumerate(zip(lens, new)):
        first, lo = _attended(case, L, n)
        if -(-first // bs) < lo // bs:
            tables[s, -(-first // bs):lo // bs] = -1
    T = sum(new) if case["op"] == "prefill" else len(lens)
    q = torch.randn((T, H * G * D), generator=g, device=DEV).to(torch.bfloat16)
    qsl = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    out = torch.empty((T, H * G, D), dtype=torch.bfloat16 if case["op"] == "prefill" else torch.float32, device=DEV)
    st.update(q=q, out=out, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), qsl=qsl,
              width=width, tokens=T, longest=max(lens), most=max(new), k_scale=1.0 / 60, v_scale=1.0 / 60)
    return st


def _layer_pools(case, g):
    """Every layer's K and V codes and their scales, each a stack of the layers' pools."""
    shape = (case["layers"], case["blocks"], case["block"], case["heads"], case["dim"])
    codes = [torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(2)]
    scales = [2.0 ** torch.randint(-9, 3, shape[:2] + shape[3:4], generator=g, device=DEV).float() for _ in range(2)]
    return codes + scales


def _prepare_fork(case, g):
    bs, nb, P, C = case["block"], case["blocks"], case["parents"], case["children"]
    lens = _parents(case)
    width = max(-(-L // bs) for L in lens) + 2
    B = P * (1 + C)
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32).cpu()
    tables = torch.full((B, width), -1, dtype=torch.int32)
    refs = torch.zeros(nb, dtype=torch.int32)
    at = 0
    for p, L in enumerate(lens):  # row p (1 + C) is parent p's; its children's rows hold the last step's forks of it
        r, full, part = p * (1 + C), L // bs, int(L % bs > 0)
        mine = perm[at:at + full + part]
        at += full + part
        tables[r, :full + part] = mine
        refs[mine.long()] = 1
        for c in range(1, 1 + C):
            tables[r + c, :full] = mine[:full]
            refs[mine[:full].long()] += 1
            if part:
                tables[r + c, full] = perm[at]
                refs[perm[at].long()] = 1
                at += 1
    seq_lens = torch.tensor(lens).repeat_interleave(1 + C).to(torch.int32)
    src = torch.arange(P).repeat_interleave(C) * (1 + C)
    dst = (torch.arange(P)[:, None] * (1 + C) + 1 + torch.arange(C)).reshape(-1)
    child = torch.zeros(B, dtype=torch.bool)
    child[dst] = True
    st = dict(op="fork", case=case, tables=tables.to(DEV), refs=refs.to(DEV), lens=seq_lens.to(DEV),
              src=src.to(torch.int32).to(DEV), dst=dst.to(torch.int32).to(DEV),
              first=torch.zeros(B, dtype=torch.int32, device=DEV),
              end=(child.to(torch.int32) * width).to(DEV), pools=_layer_pools(case, g), width=width, seqs=B,
              copy_src=torch.empty(P * C, dtype=torch.int32, device=DEV),
              copy_dst=torch.empty(P * C, dtype=torch.int32, device=DEV))
    return st


def _prepare_compact(case, g):
    nb, width, U = case["blocks"], case["max_blocks"], _used(case)
    used = torch.randperm(nb, generator=g, device=DEV)[:U].to(torch.int32).cpu()
    rows = -(-U // max(1, width - 3)) + 1
    tables = torch.full((rows, width), -1, dtype=torch.int32)
    refs = torch.zeros(nb, dtype=torch.int32)
    at = r = 0
    while at < U:
        n = min(U - at, max(1, width - 3 - (r * 5) % max(1, width // 2)))
        if r >= rows:
            tables = torch.cat([tables, torch.full((rows, width), -1, dtype=torch.int32)])
            rows = tables.shape[0]
        tables[r, :n] = used[at:at + n]
        refs[used[at:at + n].long()] = 1
        at, r = at + n, r + 1
    tables = torch.cat([tables, torch.full((1, width), -1, dtype=torch.int32)])
    share = max(1, width // 4)  # the last row shares its first pages with the first
    tables[-1, :share] = tables[0, :share]
    named = tables[0, :share]
    refs[named[named >= 0].long()] += 1
    most = max(1, nb // 2)
    e = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(op="compact", case=case, tables=tables.to(DEV), refs=refs.to(DEV), pools=_layer_pools(case, g),
                width=width, seqs=tables.shape[0], new_tables=torch.empty_like(tables, device=DEV), new_refs=e(nb),
                new_ids=e(nb), copy_src=e(most), copy_dst=e(most), num_used=e(1))


# ------------------------------------------------------------- plain forms
def _values(codes):
    return codes.view(E4M3).float() if codes.dtype == torch.uint8 else codes.float()


def _plain_write(st):
    H, D, bs = st["case"]["heads"], st["case"]["dim"], st["case"]["block"]
    T, row = st["tokens"], H * D
    lens, qsl = st["lens"].long(), st["qsl"].long()
    tok = torch.arange(T, device=DEV)
    seq = torch.searchsorted(qsl, tok, right=True) - 1
    new = qsl[1:] - qsl[:-1]
    pos = lens[seq] - new[seq] + tok - qsl[seq]
    block = st["tables"][seq, pos // bs].long()
    # sequences whose first new token falls into a block that holds earlier tokens
    kept = torch.nonzero((new > 0) & ((lens - new) % bs > 0))[:, 0]
    rows = (lens - new)[kept] % bs
    first = st["tables"][kept, (lens - new)[kept] // bs].long()
    for x, codes, scales in ((st["key"], st["kc"], st["ks"]), (st["value"], st["vc"], st["vs"])):
        x = x[:, :row].reshape(T, H, D).float()
        amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
        amax = torch.zeros_like(scales).index_reduce_(0, block, amax, "amax")
        s = _pow2_scale(amax)
        old = scales[first]
        s[first] = torch.maximum(s[first], old)
        ratio = (old / s[first])[:, None, :, None]
        c = codes[first]
        again = (_values(c) * ratio).to(E4M3).view(torch.uint8)
        keep = (torch.arange(bs, device=DEV)[None, :] < rows[:, None])[:, :, None, None]
        codes[first] = torch.where(keep, again, c)
        scales[block] = s[block]
        y = (x / s[block][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
        codes.view(-1, H, D)[block * bs + pos % bs] = y
    return _write_out(st)


def _write_out(st):
    return [st["kc"].view(E4M3), st["vc"].view(E4M3), st["ks"], st["vs"]]


def _gather(st, pos, ok):
    """K and V at positions `pos` [sequences, P] of each sequence as [sequences, heads, P, dim], zeros where not ok."""
    bs, H, D = st["case"]["block"], st["case"]["heads"], st["case"]["dim"]
    block = torch.where(ok, torch.gather(st["tables"], 1, pos // bs).long(), 0)
    slot = block * bs + torch.where(ok, pos % bs, 0)
    got = []
    for c, s, one in ((st["kc"], st["ks"], st["k_scale"]), (st["vc"], st["vs"], st["v_scale"])):
        x = _values(c.view(-1, H, D)[slot])
        if s is not None:
            x *= s[block][..., None]
        elif c.dtype == torch.uint8:
            x *= one
        got.append(torch.where(ok[..., None, None], x, 0.0).transpose(1, 2))
    return got


def _softmax_product(scores, ok, v):
    """softmax of the scores that are ok, times v; rows with none give zeros."""
    scores = torch.where(ok, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _plain_decode(st):
    case = st["case"]
    H, G, D, W, S = case["heads"], case["group"], case["dim"], case["window"], case["sinks"]
    L = st["lens"].long()[:, None]
    if W:
        start = (L - W).clamp_min(0)
        near = start + torch.arange(min(W, st["longest"]), device=DEV)
        far = torch.arange(min(S, st["longest"]), device=DEV).expand(L.shape[0], -1)
        pos, ok = torch.cat([far, near], 1), torch.cat([far < start, near < L], 1)
    else:
        pos = torch.arange(st["longest"], device=DEV).expand(L.shape[0], -1)
        ok = pos < L
    k, v = _gather(st, torch.where(ok, pos, 0), ok)
    q = st["q"].float().view(-1, H, G, D)
    scores = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
    st["out"].copy_(_softmax_product(scores, ok[:, None, None, :], v).reshape(-1, H * G, D))
    return st["out"]


def _plain_prefill(st):
    case = st["case"]
    H, G, D, W, S = case["heads"], case["group"], case["dim"], case["window"], case["sinks"]
    lens, qsl, most = st["lens"].long(), st["qsl"].long(), st["most"]
    B, T = lens.shape[0], st["tokens"]
    new = (qsl[1:] - qsl[:-1])[:, None]
    j = torch.arange(most, device=DEV)
    qpos = lens[:, None] - new + j  # [B, most]
    L = lens[:, None]
    if W:
        lo = (L - new + 1 - W).clamp_min(0)
        near = lo + torch.arange(min(W + most, st["longest"]), device=DEV)
        far = torch.arange(min(S, st["longest"]), device=DEV).expand(B, -1)
        pos, ok = torch.cat([far, near], 1), torch.cat([far < lo, near < L], 1)
    else:
        pos = torch.arange(st["longest"], device=DEV).expand(B, -1)
        ok = pos < L
    k, v = _gather(st, torch.where(ok, pos, 0), ok)
    rows = torch.where(j < new, qsl[:-1, None] + j, 0)
    q = st["q"].float().view(T, H, G, D)[rows].permute(0, 2, 3, 1, 4).reshape(B, H, G * most, D)
    scores = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
    seen = ok[:, None, :] & (pos[:, None, :] <= qpos[:, :, None])
    if W:
        seen = seen & ((pos[:, None, :] > qpos[:, :, None] - W) | (pos[:, None, :] < S))
    o = _softmax_product(scores.view(B, H, G, most, -1), seen[:, None, None], v[:, :, None])
    tok = torch.arange(T, device=DEV)
    seq = torch.searchsorted(qsl, tok, right=True) - 1
    st["out"].copy_(o.permute(0, 3, 1, 2, 4)[seq, tok - qsl[seq]].reshape(T, H * G, D))
    return st["out"]


def _plain_copy(st):
    ok = torch.nonzero(st["copy_src"] >= 0)[:, 0]
    src, dst = st["copy_src"][ok].long(), st["copy_dst"][ok].long()
    st["pools"][0][:, dst] = st["pools"][0][:, src]
    st["pools"][1][:, dst] = st["pools"][1][:, src]
    st["pools"][2][:, dst] = st["pools"][2][:, src]
    st["pools"][3][:, dst] = st["pools"][3][:, src]


def _plain_fork(st):
    bs, width, nb = st["case"]["block"], st["width"], st["case"]["blocks"]
    tables, refs, lens = st["tables"], st["refs"], st["lens"]
    src, dst = st["src"].long(), st["dst"].long()
    at = torch.arange(width, device=DEV)
    # the children's pages are let go
    gone = (at >= st["first"][:, None]) & (at < st["end"][:, None]) & (tables >= 0)
    refs -= torch.bincount(torch.where(gone, tables, nb).reshape(-1).long(), minlength=nb + 1)[:nb].to(torch.int32)
    tables.masked_fill_(gone, -1)
    # full pages are shared, a partial one gets the lowest free page, in the order of the forks
    L = lens[src].long()
    full, part = L // bs, L % bs > 0
    shared = torch.where(at < full[:, None], tables[src], -1)
    order = torch.cumsum(part, 0)
    free = torch.cumsum(refs == 0, 0)
    fresh = torch.searchsorted(free, order.clamp_min(1))
    last = torch.gather(tables[src], 1, full[:, None].clamp_max(width - 1))[:, 0]
    st["copy_src"].copy_(torch.where(part, last, -1))
    st["copy_dst"].copy_(torch.where(part, fresh, -1))
    rows = torch.where((at == full[:, None]) & part[:, None], fresh[:, None].to(torch.int32), shared)
    tables[dst] = rows
    lens[dst] = lens[src]
    refs += torch.bincount(torch.where(rows >= 0, rows, nb).reshape(-1).long(), minlength=nb + 1)[:nb].to(torch.int32)
    _plain_copy(st)
    return _fork_out(st)


def _fork_out(st):
    return [st["tables"], st["refs"], st["lens"], st["copy_src"], st["copy_dst"]] + st["pools"]


def _plain_compact(st):
    nb, refs, tables = st["case"]["blocks"], st["refs"], st["tables"]
    ids = torch.arange(nb, device=DEV)
    used = refs > 0
    count = used.sum()
    leaves, takes = used & (ids >= count), ~used & (ids < count)
    n = st["copy_src"].shape[0]
    src = torch.full((n + 1,), -1, dtype=torch.int64, device=DEV)
    dst = src.clone()
    src[torch.where(leaves, torch.cumsum(leaves, 0) - 1, n)] = ids
    dst[torch.where(takes, torch.cumsum(takes, 0) - 1, n)] = ids
    src, dst = src[:n], dst[:n]
    to = torch.where(used, ids, -1)
    to = torch.cat([to, to[:1]])
    to[torch.where(src >= 0, src, nb)] = dst
    to = to[:nb]
    st["new_ids"].copy_(to)
    spare = torch.zeros(nb + 1, dtype=torch.int32, device=DEV)
    spare[torch.where(to >= 0, to, nb)] = refs
    st["new_refs"].copy_(spare[:nb])
    st["new_tables"].copy_(torch.where(tables >= 0, to[tables.clamp_min(0).long()].to(torch.int32), -1))
    st["num_used"].copy_(count)
    st["copy_src"].copy_(src)
    st["copy_dst"].copy_(dst)
    _plain_copy(st)
    return _compact_out(st)


def _compact_out(st):
    return [st["new_tables"], st["new_refs"], st["new_ids"], st["num_used"], st["copy_src"], st["copy_dst"]] + st["pools"]


# ------------------------------------------------------- the library's calls
def _library(need=0):
    """The package, with a split-KV workspace of at least `need` bytes registered, as a server does at its start."""
    global _ws
    import paged_kv_cache_fill_gb300 as pk
    if need and (_ws is None or _ws.numel() < need):
        _ws = torch.empty(max(need, 64 << 20), dtype=torch.uint8, device=DEV)
        pk.kv_set_decode_workspace(_ws)
    return pk


def _own_write(st):
    c = st["case"]
    pk = _library()
    pk.kv_write_fp8_block(st["key"], st["value"], st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["lens"],
                          st["qsl"], st["width"], c["seqs"], st["tokens"], c["heads"], c["dim"], c["block"],
                          st["stride"], st["stride"])
    return _write_out(st)


def _own_attn(st):
    c = st["case"]
    H, D, bs, B, kind = c["heads"], c["dim"], c["block"], c["seqs"], c["kind"]
    Hq = H * c["group"]
    pk = _library()
    if st["op"] == "decode":
        pk = _library(pk.kv_decode_workspace_bytes(st["width"], B, Hq, H, D, bs))
    tail = (st["width"], B) + ((st["tokens"],) if st["op"] == "prefill" else ()) + (Hq, H, D, bs, D ** -0.5)
    lens = (st["tables"], st["lens"]) + ((st["qsl"],) if st["op"] == "prefill" else ())
    scales = {"bf16": (), "fp8k": (st["k_scale"],), "fp8": (st["k_scale"], st["v_scale"]), "fp8_block": ()}[kind]
    caches = (st["kc"], st["vc"]) + ((st["ks"], st["vs"]) if kind == "fp8_block" else ())
    name = "paged_%s_attn_%s%s" % (st["op"], kind, "" if kind == "fp8_block" else "_sinks")
    getattr(pk, name)(st["q"], *caches, st["out"], *lens, *tail, *scales, Hq * D, c["window"], c["sinks"])
    return st["out"]


def _own_copy(pk, st):
    pk.kv_copy_blocks([layer for pool in st["pools"] for layer in pool.unbind(0)], st["copy_src"], st["copy_dst"],
                      st["copy_src"].numel(), st["case"]["blocks"])


def _own_fork(st):
    c = st["case"]
    pk = _library()
    pk.kv_free_blocks(st["tables"], st["refs"], st["first"], st["end"], st["width"], st["seqs"], c["blocks"])
    pk.kv_fork_blocks(st["tables"], st["lens"], st["refs"], st["src"], st["dst"], st["copy_src"], st["copy_dst"],
                      st["src"].numel(), st["width"], st["seqs"], c["blocks"], c["block"])
    _own_copy(pk, st)
    return _fork_out(st)


def _own_compact(st):
    c = st["case"]
    pk = _library()
    pk.kv_compact_blocks(st["tables"], st["refs"], st["new_tables"], st["new_refs"], st["new_ids"], st["copy_src"],
                         st["copy_dst"], st["num_used"], st["width"], st["seqs"], c["blocks"])
    _own_copy(pk, st)
    return _compact_out(st)


def run(state):
    if own:
        return {"write": _own_write, "decode": _own_attn, "prefill": _own_attn, "fork": _own_fork,
                "compact": _own_compact}[state["op"]](state)
    return {"write": _plain_write, "decode": _plain_decode, "prefill": _plain_prefill, "fork": _plain_fork,
            "compact": _plain_compact}[state["op"]](state)


# ----------------------------------------------------------------- 64 bits
def _e4m3_64(codes):
    """E4M3 codes' values from their bits: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = codes.to(torch.int32)
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e.double() - 7))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def _scale_64(amax):
    a = amax / E4M3_MAX
    s = torch.ones_like(a)
    up = torch.ceil(torch.log2(torch.where(a > 0, a, s)))
    up = torch.where(2.0 ** (up - 1) >= a, up - 1, up)
    up = torch.where(2.0 ** up < a, up + 1, up)
    return torch.where(a > 0, 2.0 ** up, 0.0).clamp_min(MIN_SCALE)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None  # whole numbers and copies
    flops = work(case)["flops"]
    if flops > 3e12:
        return None
    st = prepare(case, seed)
    return _exact_write(st) if op == "write" else _exact_attn(st)


def _exact_write(st):
    """The stored values before their rounding to 8 bits, and the scales."""
    case = st["case"]
    H, D, bs = case["heads"], case["dim"], case["block"]
    lens, qsl, tables = st["lens"].tolist(), st["qsl"].tolist(), st["tables"].cpu()
    got = []
    for x, codes, scales in ((st["key"], st["kc"], st["ks"]), (st["value"], st["vc"], st["vs"])):
        vals = _e4m3_64(codes)
        new_scales = scales.double()
        for s, L in enumerate(lens):
            n = qsl[s + 1] - qsl[s]
            rows = x[qsl[s]:qsl[s + 1], :H * D].double().view(n, H, D)
            p = L - n
            while p < L:
                b = int(tables[s, p // bs])
                end = min(L, (p // bs + 1) * bs)
                y = rows[p - (L - n):end - (L - n)]
                want = _scale_64(y.abs().amax((0, 2)))
                if p % bs:
                    was = new_scales[b].clone()
                    want = torch.maximum(want, was)
                    vals[b, :p % bs] *= (was / want)[:, None]
                new_scales[b] = want
                vals[b, p % bs:p % bs + end - p] = y / want[:, None]
                p = end
        got += [vals, new_scales]
    return [got[0], got[2], got[1], got[3]]


def _exact_attn(st):
    case = st["case"]
    H, G, D, bs, W, S = (case[x] for x in ("heads", "group", "dim", "block", "window", "sinks"))
    lens, qsl = st["lens"].tolist(), st["qsl"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for s, L in enumerate(lens):
        n = qsl[s + 1] - qsl[s] if st["op"] == "prefill" else 1
        r0 = qsl[s] if st["op"] == "prefill" else s
        if L == 0 or n == 0:
            continue
        first, lo = _attended(case, L, n)
        pos = torch.cat([torch.arange(0, first, device=DEV), torch.arange(lo, L, device=DEV)])
        b = st["tables"][s].long()[pos // bs]
        kv = []
        for c, sc, one in ((st["kc"], st["ks"], st["k_scale"]), (st["vc"], st["vs"], st["v_scale"])):
            x = c[b, pos % bs]
            if c.dtype == torch.uint8:
                x = _e4m3_64(x) * (sc[b].double()[..., None] if sc is not None else one)
            kv.append(x.double().transpose(0, 1))  # [H, P, D]
        at = torch.arange(L - n, L, device=DEV)[:, None]
        seen = pos <= at
        if W:
            seen &= (pos > at - W) | (pos < S)
        step = max(1, (1 << 27) // (H * G * pos.numel()))
        for j in range(0, n, step):
            m = min(step, n - j)
            q = st["q"][r0 + j:r0 + j + m].double().view(m, H, G, D).permute(1, 2, 0, 3).reshape(H, G * m, D)
            z = (q @ kv[0].transpose(1, 2)).view(H, G, m, -1) / math.sqrt(D)
            z = z.masked_fill(~seen[j:j + m], -math.inf)
            p = torch.softmax(z, -1).view(H, G * m, -1)
            out[r0 + j:r0 + j + m] = (p @ kv[1]).view(H, G, m, D).permute(2, 0, 1, 3).reshape(m, H * G, D)
    return out
