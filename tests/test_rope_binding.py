"""What the binding of the rotations does by itself, on the CPU."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALL = """
import paged_kv_cache_fill_gb300 as pk
try:
    pk.kv_rope_frequencies(%d, 10000.0)
except pk.PagedKVError as e:
    print("status", e.status)
"""


@pytest.mark.parametrize("rotary_dim", [-2, -128, -1, -2 ** 31, 2 ** 32 + 8, 2 ** 32, 0, 7])
def test_frequencies_of_no_dim(rotary_dim):
    """Refused before anything is allocated or written (in a process of its own: the array lies on the heap)."""
    from paged_kv_cache_fill_gb300 import _build
    _build.build()
    r = subprocess.run([sys.executable, "-c", CALL % rotary_dim], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["status", "1"], (r.returncode, r.stdout, r.stderr[-500:])
