"""The bounds-checking build with the block-scaled cache: a block id past the
pool is flagged, its rows are not written, and attention reads block 0 (and
its scales) in its place; what does not use it is untouched."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KV_OK, KV_ERR_DEVICE, BIT_OUT_OF_POOL = 0, 4, 8


def test_block_scaled_calls_flag_ids_past_the_pool():
    sys.path.insert(0, os.path.join(ROOT, "paged_kv_cache_fill_gb300"))
    import _build
    library = _build.build(debug=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_block_child.py"), library],
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["clean"] == [KV_OK, 0]
    for step in ("write", "decode", "prefill"):
        assert res[step] == [KV_ERR_DEVICE, BIT_OUT_OF_POOL], (step, res[step])
    assert res["write_equal"] and res["prefill_finite"]
    # |v| < 6 and sums of |q k| / sqrt(128) below 16: 2 * 6 * (136 * 2^-23 * 16 + 2^-20)
    assert res["decode_err"] <= 3.2e-3, res
