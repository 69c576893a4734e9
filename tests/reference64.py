"""Plain 64-bit references of the block-scaled FP8 write, of attention with a
sliding window and sinks, and of the page calls, in numpy on the CPU: one
sequence, one head, one page at a time, straight from the definitions."""
import numpy as np
import torch

E4M3_MAX, MIN_SCALE = 448.0, 2.0 ** -60


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """E4M3 codes -> float64 (sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7F / 0xFF NaN)."""
    c = codes.astype(np.int64)
    e, f = (c >> 3) & 15, (c & 7) / 8.0
    v = np.where(e == 0, f * 2.0 ** -6, (1 + f) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """float64 -> E4M3 codes, round to nearest even, saturating; NaN 0x7F. The value is first rounded to a
    multiple of the format's step at its magnitude, which the conversion then holds exactly."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x)
    a = np.clip(np.where(nan, 0.0, x), -E4M3_MAX, E4M3_MAX)
    step = 2.0 ** (np.maximum(np.frexp(np.abs(a))[1] - 1, -6) - 3)
    a = np.clip(np.rint(a / step) * step, -E4M3_MAX, E4M3_MAX)
    a = np.where(a == 0, np.copysign(0.0, np.where(nan, 0.0, x)), a)
    c = torch.from_numpy(a.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.where(nan, 0x7F, c).astype(np.uint8)


def pow2_scale(amax: float) -> float:
    s = MIN_SCALE
    while amax > E4M3_MAX * s:
        s *= 2.0
    return s


def write_block(key, value, codes, scales, tables, lens, qsl, H, D, bs):
    """key, value float64 [tokens, >= H D] arrays; codes (K, V) uint8 [blocks, bs, H, D] and scales (K, V) float32
    [blocks, H], updated in place."""
    cap = tables.shape[1] * bs
    for x, c, sc in ((key, codes[0], scales[0]), (value, codes[1], scales[1])):
        for s in range(len(lens)):
            n, L = int(qsl[s + 1] - qsl[s]), int(lens[s])
            begin, end = max(0, L - n), min(L, cap)
            for lb in range(begin // bs, -(-end // bs) if end > begin else begin // bs):
                p0, p1 = max(begin, lb * bs), min(end, (lb + 1) * bs)
                b = int(tables[s, lb])
                if b < 0 or p0 >= p1:
                    continue
                tok = int(qsl[s]) + p0 - (L - n)
                new = x[tok:tok + p1 - p0, :H * D].reshape(-1, H, D)
                r0 = p0 - lb * bs
                for h in range(H):
                    y = new[:, h]
                    fin = np.abs(y[np.isfinite(y)])
                    s1 = pow2_scale(fin.max() if fin.size else 0.0)
                    if r0:
                        s0 = float(sc[b, h])
                        if s0 >= s1:
                            s1 = s0
                        else:
                            c[b, :r0, h] = e4m3_codes(e4m3_values(c[b, :r0, h]) * (s0 / s1))
                    sc[b, h] = s1
                    c[b, r0:r0 + p1 - p0, h] = e4m3_codes(y / s1)


def attended(P: int, W: int, S: int) -> np.ndarray:
    """Positions that a query at position P attends."""
    p = np.arange(P + 1)
    return p if W == 0 else p[(p > P - W) | (p < S)]


def attention(q, k, v, P, W, S, scale):
    """One query q [D] at position P over the rows k, v of a sequence (float64, indexed by position): output [D],
    the largest |v| it saw, and the largest sum |q k| scale; zeros if it attends nothing."""
    pos = attended(P, W, S) if P >= 0 else np.zeros(0, np.int64)
    if pos.size == 0:
        return np.zeros(v.shape[1]), 0.0, 0.0
    z = k[pos] @ q * scale
    w = np.exp(z - z.max())
    return (w / w.sum()) @ v[pos], np.abs(v[pos]).max(), (np.abs(k[pos]) @ np.abs(q)).max() * abs(scale)


def free_blocks(tables, refs, first, end):
    for s in range(tables.shape[0]):
        for j in range(max(0, int(first[s])), min(int(end[s]), tables.shape[1])):
            b = int(tables[s, j])
            if b >= 0:
                tables[s, j] = -1
                if b < len(refs) and refs[b] > 0:
                    refs[b] -= 1


def fork_blocks(tables, lens, refs, src, dst, bs):
    """Returns (copy_src, copy_dst)."""
    B, width = tables.shape
    valid = lambda r: 0 <= r < B  # noqa: E731
    pages = []
    for s, d in zip(src, dst):
        ok = valid(s) and valid(d) and list(dst).count(d) == 1 and s not in list(dst) and 0 <= lens[s] <= width * bs
        page = -2
        if ok:
            page = int(tables[s, lens[s] // bs]) if lens[s] % bs else -1
            page = -1 if page < 0 else page if page < len(refs) else -2
        pages.append(page)
    free = [b for b in range(len(refs)) if refs[b] <= 0]
    pairs = []
    for page in pages:
        if page < 0:
            pairs.append((page, page))
        elif free:
            pairs.append((page, free.pop(0)))
            refs[pairs[-1][1]] = 1
        else:
            pairs.append((-2, -2))
    for (s, d), (_, fresh) in zip(zip(src, dst), pairs):
        if fresh == -2:
            continue
        full = int(lens[s]) // bs
        row = np.full(width, -1, tables.dtype)
        for j in range(full):
            b = int(tables[s, j])
            if 0 <= b < len(refs):
                row[j] = b
                refs[b] += 1
        if full < width:
            row[full] = fresh
        tables[d], lens[d] = row, lens[s]
    return np.array([p[0] for p in pairs], np.int32), np.array([p[1] for p in pairs], np.int32)


def compact_blocks(tables, refs):
    """Returns (tables, refs, ids, copy_src, copy_dst, used)."""
    n = len(refs)
    used = [b for b in range(n) if refs[b] > 0]
    U = len(used)
    src = [b for b in used if b >= U]
    dst = [b for b in range(U) if refs[b] <= 0]
    ids = np.full(n, -1, np.int32)
    ids[used] = used
    ids[src] = dst
    out = np.zeros(n, np.int32)
    for b in used:
        out[ids[b]] = refs[b]
    t = np.where((tables >= 0) & (tables < n), ids[np.clip(tables, 0, n - 1)], -1).astype(np.int32)
    pad = [-1] * (n // 2 - len(src))
    return t, out, ids, np.array(src + pad, np.int32), np.array(dst + pad, np.int32), U
