"""A split decode whose pipeline waits give up: the count of pieces that each
sequence was cut into, which the combine kernel reads from the workspace, is
written all the same, so that nothing a call reads there is left from before.
In the bounds-checking build, whose wait limit can be cut to 1 ns (every wait
is bounded, and no access leaves the buffers)."""
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
BIT_TIMEOUT = 1


def test_piece_counts_are_written_by_a_decode_that_gave_up():
    sys.path.insert(0, os.path.join(ROOT, "paged_kv_cache_fill_gb300"))
    import _build
    library = _build.build(debug=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "decode_timeout_child.py"), library],
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    for kind in ("fp8k", "fp8_block"):
        assert res[kind]["clean"] == 0 and res[kind]["bits"] == BIT_TIMEOUT, res
        assert res[kind]["wrong_counts"] == 0, res
        assert res[kind]["after"] == 0 and res[kind]["same"], res
