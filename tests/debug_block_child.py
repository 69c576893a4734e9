"""Child process of tests/test_block_debug_gpu.py: loads the bounds-checking
library alone and runs the block-scaled write, decode and prefill with a block
table that holds one id past the pool; prints its findings as one JSON line.
Every buffer has the size that the good ids need, and the bad one is never
dereferenced. Run: python tests/debug_block_child.py <library path>"""
import ctypes
import json
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]

import paged_kv_cache_fill_gb300 as pk  # noqa: E402
import reference64 as ref  # noqa: E402

DEV = torch.device("cuda")


def status():
    bits = ctypes.c_uint32(0)
    return [int(pk.lib().kv_get_device_error(ctypes.byref(bits))), int(bits.value)]


def main(path):
    pk.use_library(path)
    rng = np.random.default_rng(2)
    H, Hq, D, bs, nb = 2, 4, 128, 16, 8
    lens = np.array([40, 33])
    tables = np.array([[0, 1, 2], [3, nb + 5, 4]], np.int32)      # sequence 1's second block is no block
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    res = {"clean": status()}
    assert pk.lib().kv_debug_set_pool(nb, bs) == pk.KV_OK
    codes = [np.full((nb, bs, H, D), 0x7F, np.uint8) for _ in range(2)]
    scales = [np.full((nb, H), 1.0, np.float32) for _ in range(2)]
    dc, ds = [torch.from_numpy(c).to(DEV) for c in codes], [torch.from_numpy(s).to(DEV) for s in scales]
    T = int(lens.sum())
    x = [torch.from_numpy(rng.standard_normal((T, H * D)).astype(np.float32)).to(torch.bfloat16) for _ in range(2)]
    qsl = [0, 40, 73]
    pk.kv_write_fp8_block(x[0].to(DEV), x[1].to(DEV), *dc, *ds, i32(tables), i32(lens), i32(qsl), 3, 2, T, H, D, bs, H * D,
                          H * D)
    res["write"] = status()
    skip = tables.copy()
    skip[1, 1] = -1
    ref.write_block(x[0].double().numpy(), x[1].double().numpy(), codes, scales, skip, lens, qsl, H, D, bs)
    res["write_equal"] = all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(dc + ds, codes + scales))
    q = torch.from_numpy(rng.standard_normal((T, Hq * D)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    out = torch.zeros((2, Hq, D), device=DEV)
    pk.paged_decode_attn_fp8_block(q, *dc, *ds, out, i32(tables), i32(lens), 3, 2, Hq, H, D, bs, D ** -0.5, Hq * D, 0, 0)
    res["decode"] = status()
    pre = torch.zeros((T, Hq, D), device=DEV, dtype=torch.bfloat16)
    pk.paged_prefill_attn_fp8_block(q, *dc, *ds, pre, i32(tables), i32(lens), i32(qsl), 3, 2, T, Hq, H, D, bs, D ** -0.5,
                                    Hq * D, 0, 0)
    res["prefill"] = status()
    # sequence 0 does not use the bad block
    k, v = (ref.e4m3_values(codes[i][tables[0]].reshape(-1, H, D)[:40])
            * scales[i][tables[0]].repeat(bs, 0)[:40].astype(np.float64)[..., None] for i in range(2))
    err = 0.0
    for h in range(Hq):
        o, _, _ = ref.attention(q[0].double().cpu().numpy()[h * D:(h + 1) * D], k[:, h // 2], v[:, h // 2], 39, 0, 0,
                                D ** -0.5)
        err = max(err, float(np.abs(out[0, h].double().cpu().numpy() - o).max()))
    res["decode_err"] = err
    res["prefill_finite"] = bool(torch.isfinite(pre[:40].float()).all())
    print(json.dumps(res))


main(sys.argv[1])
