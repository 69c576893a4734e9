"""Refusals of the float-row chunked prefills that test_abi.py does not cover (no GPU needed)."""
import pytest

from test_operators_abi import FAKE, pk  # noqa: F401 - the library as a fixture


@pytest.mark.parametrize("kind,scales", [("bf16", []), ("fp8k", [1.0]), ("fp8", [1.0, 1.0])])
def test_prefill_refuses_negative_score_scales(pk, kind, scales):  # noqa: F811
    call = getattr(pk.lib(), f"paged_prefill_attn_{kind}")
    for isd in (-0.1, -1e-38, float("-inf")):
        assert call(*[FAKE] * 7, 4, 2, 10, 32, 8, 128, 16, isd, *scales, 4096, 0, None) == pk.KV_ERR_INVALID_ARG
    # nothing to do: not looked at, as with the other arguments
    assert call(*[None] * 7, 4, 0, 10, 32, 8, 128, 16, -0.1, *scales, 4096, 0, None) == pk.KV_OK
