"""Rotary positions beside values that are not finite, with the references and
tolerances of test_rope_gpu.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_fill_gb300 as pk
import rope64
from test_rope_gpu import DEV, check_bf16, f64, i32, table

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_finite_pairs_beside_a_non_finite_one(bad, interleaved, inverse):
    """A pair's result does not depend on its neighbours: every finite pair, near-cancelling ones, beside one that holds an
    infinity or a NaN gives the bits that it gives without it."""
    T, D = 64, 64
    freqs, tab = table(D)
    pos = np.arange(T) * 1237 + 5
    th = rope64.angles(pos, freqs)
    i = np.arange(D // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + D // 2)
    x = np.empty((T, D))
    x[:, a], x[:, b] = np.sin(th), np.cos(th) * (-1 if inverse else 1)
    x = torch.from_numpy(x).to(torch.bfloat16)
    y = x.clone()
    hit = (np.arange(T) * 5) % (D // 2)  # the pair of each row
    at = np.where(np.arange(T) % 2, a[hit], b[hit])
    y[np.arange(T), at] = bad
    out = [torch.empty_like(x, device=DEV) for _ in range(2)]
    for src, dst in zip((x, y), out):
        pk.kv_rope(src.to(DEV), dst, tab, i32(pos), T, 1, D, D, D, D, interleaved, inverse)
    clean, got = (o.cpu() for o in out)
    pair = torch.zeros((T, D), dtype=torch.bool)
    pair[np.arange(T), a[hit]] = pair[np.arange(T), b[hit]] = True
    assert torch.equal(got[~pair].view(torch.int16), clean[~pair].view(torch.int16))
    assert not torch.isfinite(got[pair].float()).any()
    if bad == bad:  # (no sine or cosine is zero here)
        assert torch.isinf(got[pair].float()).all()
    want, mag = rope64.rotate(f64(x)[:, None], pos, freqs, 1.0, interleaved, inverse)
    check_bf16(f64(clean)[:, None], want, mag)
