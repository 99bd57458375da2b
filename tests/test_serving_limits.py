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


def test_workspace_holds_two_partials_a_column():
    """Per column two partials of every head (dv sums; reference and denominator) and one entry of 16 bytes, each array padded to
    256 bytes; 152 SMs of two CTAs over bf16 and up to three over E4M3, whichever needs more; nothing for a single column."""
    def columns(kv_heads, ctas):
        best, fullest = 1, 0.0
        for waves in range(1, 5):
            c = waves * 152 * ctas // kv_heads
            if c and c * kv_heads / (waves * 152 * ctas) > fullest + 1e-9:
                best, fullest = c, c * kv_heads / (waves * 152 * ctas)
            if fullest >= 0.96:
                break
        return best

    def padded(n):
        return (n + 255) // 256 * 256

    for heads, kv_heads, dq, dv, ctas in ((8, 2, 128, 128, 3), (64, 8, 128, 128, 3), (12, 12, 192, 128, 2), (5, 5, 64, 64, 3), (128, 128, 64, 128, 3)):
        c = max(columns(kv_heads, 2), columns(kv_heads, ctas))
        want = padded(c * 2 * heads * dv * 4) + padded(c * 2 * heads * 8) + padded(c * 16)
        assert vpp.decode_attn_workspace_size(3, heads, kv_heads, dq, dv) == want
    assert vpp.decode_attn_workspace_size(3, 1024, 1024, 64, 64) == 0


def test_host_tensors_are_refused_by_name(lib):  # noqa: F811
    """A tensor that is not on the device of the call: the refusal says which."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    cu, bt = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1), dtype=torch.int32)
    c = vpp._calls()
    with pytest.raises(ValueError, match="q must be on the current CUDA device"):
        c.prompt(0, 0, x, x, x, cu, x, None, 0.0)
    kc = torch.zeros((1, 64, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache must be on the current CUDA device"):
        c.decode(0, 0, x, kc, kc, None, None, bt, cu, x, None, 0.0, 0, 0)
    with pytest.raises(ValueError, match="k must be on the current CUDA device"):
        c.rope(0, 0, x, x, x, None, kc, kc, None, None, bt, cu, None, x, None, 0, False)
