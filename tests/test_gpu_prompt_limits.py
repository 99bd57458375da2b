"""Packed prompt attention at the edges of what its values and neighbours may be."""

import math

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, attend, check_attention, randn
from tests.test_gpu_prompt import LENS, SHAPES, check_sequences, starts, views

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


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,Hkv,dq,dv", [(32, 8, 128, 128), (20, 20, 192, 128), (12, 1, 192, 64), (5, 1, 64, 128), (8, 8, 64, 64), (26, 2, 128, 64)])
def test_hostile_neighbours_of_long_sequences(H, Hkv, dq, dv, bad):
    """Sequences of many key tiles with partial last ones, several items a CTA, hostile values before, between and behind them."""
    lens = [40, 700, 1, 1500, 130, 300, 129, 385, 64, 1027, 5]
    good = [1, 3, 5, 7, 9]
    cu = starts(lens)
    T = int(cu[-1]) + 77
    q, k, v = randn((T, H, dq), 4), randn((T, Hkv, dq), 5), randn((T, Hkv, dv), 6)
    live = torch.zeros(T, dtype=torch.bool)
    for b in good:
        live[int(cu[b]):int(cu[b + 1])] = True
    for x in (q, k, v):
        x[~live] = bad
    lse = torch.empty((H, T), device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse)
    assert vpp.vpp_last_device_status() == 0
    for b in good:
        lo, hi = int(cu[b]), int(cu[b + 1])
        ref = attend(q[lo:hi], k[lo:hi], v[lo:hi], dq ** -0.5, True)
        check_attention(out[lo:hi], lse[:, lo:hi], ref, dq, HALF_BF16, f"sequence {b}")


@pytest.mark.parametrize("H,Hkv,lens", [(1024, 1024, [3, 200]), (2048, 1024, [70, 1]), (1000, 500, [33, 129])])
def test_many_kv_heads(H, Hkv, lens):
    d = 64
    cu = starts(lens)
    T = int(cu[-1])
    q, k, v = randn((T, H, d), 7), randn((T, Hkv, d), 8), randn((T, Hkv, d), 9)
    lse = torch.empty((H, T), device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse)
    assert vpp.vpp_last_device_status() == 0
    for b, n in enumerate(lens):
        lo, hi = int(cu[b]), int(cu[b]) + n
        ref = attend(q[lo:hi], k[lo:hi], v[lo:hi], d ** -0.5, True)
        check_attention(out[lo:hi], lse[:, lo:hi], ref, d, HALF_BF16, f"sequence {b}")


def test_a_hundred_thousand_sequences_mostly_empty():
    H, Hkv, d = 4, 2, 64
    lens = [0] * 100000
    for i, n in ((0, 3), (127, 1), (128, 200), (50000, 17), (99999, 90)):
        lens[i] = n
    cu = starts(lens)
    T = int(cu[-1])
    q, k, v = randn((T, H, d), 10), randn((T, Hkv, d), 11), randn((T, Hkv, d), 12)
    lse = torch.empty((H, T), device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse)
    assert vpp.vpp_last_device_status() == 0
    for lo, hi in sorted({(int(a), int(b)) for a, b in zip(cu, cu[1:]) if b > a}):
        ref = attend(q[lo:hi], k[lo:hi], v[lo:hi], d ** -0.5, True)
        check_attention(out[lo:hi], lse[:, lo:hi], ref, d, HALF_BF16, f"rows {lo} to {hi}")


def test_the_cached_path_gives_the_same_attention():
    """The packed call and the host-planned call over a paged cache: each is within its own distance of the formula, so they are
    within both of each other."""
    H, Hkv, d, n = 16, 4, 128, 700
    q, k, v = (randn((n, h, d), 14 + h) for h in (H, Hkv, Hkv))
    cu = torch.tensor([0, n], dtype=torch.int32)
    table = torch.arange((n + 63) // 64, dtype=torch.int32, device=DEV)[None]
    kc = torch.zeros((table.shape[1], 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    vpp.vpp_kv_append_varlen(k.to(DEV), v.to(DEV), kc, vc, table, cu.numpy(), [n])
    a = vpp.vpp_mixed_attn(q.to(DEV), kc, vc, table, cu.numpy(), [n]).double().cpu()
    b = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV)).double().cpu()
    o, _, absw, _ = attend(q, k, v, d ** -0.5, True)
    # each side: P to bf16, one rounding of the result to bf16 (see check_attention; 2^-14 holds its float32 terms at these sizes)
    tol = 2 * (HALF_BF16 * o.abs() + (HALF_BF16 + 2.0 ** -14) * absw)
    assert bool(((a - b).abs() <= tol).all())


@pytest.mark.parametrize("lens,rest", [(LENS + [0] * 4, 0), ([77, 20, 130, 1], 300), ([96] * 40, 0), ([97] * 40, 0), ([128] * 30, 0)])
@pytest.mark.parametrize("H,Hkv,dq,dv", SHAPES + [(32, 8, 128, 128), (21, 7, 64, 128), (32, 8, 64, 64)])
def test_both_forms(H, Hkv, dq, dv, lens, rest):
    """Batches on both sides of the choice between one query tile a CTA and pairs of tiles."""
    cu = starts(lens)
    T = int(cu[-1]) + rest
    x = randn((T, H * dq + Hkv * (dq + dv)), 13)
    lse = torch.full((H, T), 7.0, device=DEV)
    out = torch.full((T, H, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    vpp.vpp_prompt_attn(*views(x.to(DEV), H, Hkv, dq, dv), cu.to(DEV), out=out, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_sequences(out, lse, *views(x, H, Hkv, dq, dv), cu, dq)
    assert bool((out[int(cu[-1]):] == 7).all()) and bool((lse[:, int(cu[-1]):] == 7).all())
