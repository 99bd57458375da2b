"""Packed prompt attention at the edges of what its values and neighbours may be."""

import math

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, attend, check_attention, randn
from tests.test_gpu_prompt import starts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H,Hkv,dq,dv,lens", [(4, 2, 64, 64, [40, 3]), (32, 8, 128, 128, [1, 700, 260]), (6, 6, 192, 128, [300, 20])])
def test_rows_whose_scores_are_all_minus_infinity(H, Hkv, dq, dv, lens):
    """Finite queries and keys whose products leave float32: the weights of such a row sum to nothing, out = 0 and lse = -inf as
    for an empty row of decode; rows that see one finite score have it alone; the other heads are untouched."""
    cu = starts(lens)
    T = int(cu[-1])
    q, k, v = randn((T, H, dq), 1), randn((T, Hkv, dq), 2), randn((T, Hkv, dv), 3)
    G = H // Hkv
    q[:, :G], k[:, 0] = 0, 0
    q[:, :G, 0], k[:, 0, 0] = 2.0e38, -2.0e38
    at = int(cu[-2]) + lens[-1] // 2  # in the last sequence one key of kv head 0 has a finite score
    k[at, 0, 0] = 0.0
    lse = torch.full((H, T), 7.0, device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse).float().cpu()
    assert vpp.vpp_last_device_status() == 0
    lse = lse.cpu()
    assert not bool(out[:at, :G].any()) and bool((lse[:G, :at] == -math.inf).all())
    assert torch.equal(out[at:, :G], v[at, 0].float().expand(T - at, G, dv)) and bool((lse[:G, at:] == 0).all())
    for b, n in enumerate(lens):
        lo, hi = int(cu[b]), int(cu[b]) + n
        ref = attend(q[lo:hi, G:], k[lo:hi, 1:], v[lo:hi, 1:], dq ** -0.5, True)
        check_attention(out[lo:hi, G:], lse[G:, lo:hi], ref, dq, HALF_BF16, f"sequence {b}")
