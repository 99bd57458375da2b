"""Limits of the device-planned serving operators that the host checks before any launch."""

import pytest

from chunked_prefill_causal_gb300 import vpp
from tests.test_serving_abi import DEC, INV, P, PRO, ROPE, args, lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("batch", [1 << 30, (1 << 31) - 1])
def test_batches_beyond_the_index_arithmetic_are_refused(lib, batch):  # noqa: F811
    """A search over 2^30 sequences would add two 31-bit indexes in 32 bits and read in front of the array."""
    rope = args(ROPE, dict(batch=batch))
    assert lib.vpp_rope_append(*rope) == INV
    at = list(ROPE).index("bt")
    assert lib.vpp_rope_append_fp8(*rope[:at], P, P, *rope[at:]) == INV
    dec = args(DEC, dict(batch=batch, mb=1))
    assert lib.vpp_decode_attn(*dec) == INV
    assert lib.vpp_decode_attn_fp8(*dec[:4], P, P, *dec[4:]) == INV
    assert lib.vpp_prompt_attn(*args(PRO, dict(batch=batch))) == INV
    assert vpp.decode_attn_workspace_size(batch, 8, 2, 128, 128) == 0
