"""The Python binding's own work, on the CPU: what it hands to the C library, and
which tensors it refuses."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import paged_kv_cache_fill_gb300 as pk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class FakeLibrary:
    """Records each call's arguments; every call succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name == "kv_copy_blocks":  # the arrays live as long as the call
                args = ([int(x) for x in (ctypes.c_uint64 * args[2]).from_address(args[0])],
                        [int(x) for x in (ctypes.c_uint64 * args[2]).from_address(args[1])], *args[2:])
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    """A library that records, and a binding that refuses no tensor of the host."""
    library = FakeLibrary()
    monkeypatch.setattr(pk, "_lib", library)
    monkeypatch.setattr(pk, "_device", lambda: -1)
    monkeypatch.setattr(pk, "_refuse", lambda t: None)
    return library


@pytest.mark.parametrize("form", [list, tuple, iter, lambda pools: (p for p in pools), lambda pools: dict(
    enumerate(pools)).values()])
def test_copy_blocks_hands_over_every_pool(fake, form):
    pools = [torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2), torch.zeros(4, 8, 3, dtype=torch.bfloat16)]
    ids = torch.zeros(1, dtype=torch.int32)
    pk.kv_copy_blocks(form(pools), ids, ids, 1, 4, stream=0)
    (name, args), = fake.calls
    assert name == "kv_copy_blocks" and args[2] == 3
    assert args[0] == [p.data_ptr() for p in pools] and args[1] == [64, 8, 48]


def test_host_tensors_are_refused_with_and_without_a_gpu():
    t = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: pk.kv_copy_blocks([t], t, t, 1, 4, stream=0),
                 lambda: pk.kv_free_blocks(t, t, t, t, 1, 1, 4, stream=0),
                 lambda: pk.kv_fill_slots(t, t, 0, 4, 16, stream=0),
                 lambda: pk.kv_fork_blocks(t, t, t, t, t, t, t, 1, 1, 4, 4, 16, stream=0)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_an_empty_host_tensor_passes(monkeypatch):
    """It is never read: a call without work takes it, with and without a GPU."""
    library = FakeLibrary()
    monkeypatch.setattr(pk, "_lib", library)
    t = torch.zeros(0, dtype=torch.int32)
    pk.kv_free_blocks(t, t, t, t, 1, 0, 4, stream=0)
    assert library.calls[-1][1][:4] == (None,) * 4


def test_import_without_cuda_in_torch():
    """A torch built without CUDA lacks the names that this module takes from torch._C."""
    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import paged_kv_cache_fill_gb300 as pk\n"
            "try:\n    pk.kv_fill_slots(torch.zeros(1), torch.zeros(1), 0, 1, 16, stream=0)\n"
            "except ValueError: print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]
