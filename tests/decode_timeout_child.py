"""Child process of tests/test_decode_timeout_gpu.py: loads the bounds-checking
library alone and runs split decodes whose pipeline waits give up after 1 ns,
over a workspace filled with ones' bits; prints its findings as one JSON line.
Run: python tests/decode_timeout_child.py <library path>"""
import json
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]

import paged_kv_cache_fill_gb300 as pk  # noqa: E402

DEV = torch.device("cuda")
HEADER = 256                     # bytes of the workspace before the piece counts


def pieces(lens, head_groups, ctas, least):
    """Pieces of each (sequence, head group): the tiles of all of them in one stream, cut into equal chunks of at least
    `least` tiles."""
    tiles = [-(-int(L) // 16) for L in lens]
    total = sum(tiles) * head_groups
    chunk = max(-(-total // ctas), least)
    out, a = [], 0
    for t in tiles:
        for _ in range(head_groups):
            out.append((a + t - 1) // chunk - a // chunk + 1 if t else None)
            a += t
    return out


def case(kind, lens, H, group, D):
    bs, Hq = 16, H * group
    blocks = [-(-int(L) // bs) for L in lens]
    width, nb = max(blocks), sum(blocks)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(blocks):
        tables[s, :n] = torch.arange(at, at + n)
        at += n
    g = torch.Generator(device=DEV).manual_seed(5)
    codes = [torch.randint(0, 100, (nb, bs, H, D), generator=g, device=DEV, dtype=torch.uint8) for _ in range(2)]
    v16 = torch.randn((nb, bs, H, D), generator=g, device=DEV).to(torch.bfloat16)
    scales = [torch.full((nb, H), 2.0 ** -7, device=DEV) for _ in range(2)]
    q = torch.randn((len(lens), Hq * D), generator=g, device=DEV).to(torch.bfloat16)
    out = torch.empty((len(lens), Hq, D), device=DEV)
    tables, seq_lens = tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    geo = [width, len(lens), Hq, H, D, bs, D ** -0.5]
    ws = torch.empty(pk.kv_decode_workspace_bytes(*geo[:-1]), dtype=torch.uint8, device=DEV)
    pk.kv_set_decode_workspace(ws)

    def decode():
        if kind == "fp8k":
            pk.paged_decode_attn_fp8k(q, codes[0], v16, out, tables, seq_lens, *geo, 2.0 ** -7, Hq * D, 0)
        else:
            pk.paged_decode_attn_fp8_block(q, *codes, *scales, out, tables, seq_lens, *geo, Hq * D, 0, 0)
        return pk.kv_get_device_error()
    res = {"clean": decode()}
    want = out.clone()
    pk.kv_debug_set_wait_limit(1)
    res["bits"], res["wrong_counts"] = 0, 0
    for _ in range(8):
        ws.fill_(0x7F)           # a count of 2,139,062,143 pieces wherever the call writes none
        res["bits"] |= decode()
        # the workspace holds the pieces of chunks of 16 tiles; 8 heads to a group (groups of at most 8 query heads);
        # FP8 K and V at this size: two CTAs to an SM
        expect = pieces(lens, -(-H // 8), pk.kv_device_info()[0] * (1 if kind == "fp8k" else 2), 16)
        got = ws[HEADER:HEADER + 4 * len(expect)].view(torch.int32).tolist()
        res["wrong_counts"] += sum(e is not None and e != n for e, n in zip(expect, got))
        if res["bits"]:
            break
    pk.kv_debug_set_wait_limit(0)
    res["after"] = decode()
    res["same"] = bool(torch.equal(out, want))
    pk.kv_set_decode_workspace(None)
    return res


def main(path):
    pk.use_library(path)
    torch.cuda.set_device(0)
    rng = np.random.default_rng(1)
    lens = [6000, 30, 0, 9000, 100, 4500] + [int(x) for x in rng.integers(0, 400, 60)]
    print(json.dumps({kind: case(kind, lens, 8, 4, 128) for kind in ("fp8k", "fp8_block")}))


main(sys.argv[1])
