"""The Python binding's own work, on the CPU: what it hands to the C library, and
which tensors it refuses."""
import ctypes

import pytest
import torch

import paged_kv_cache_fill_gb300 as pk


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
