"""Packed prompt attention against the formula in 64 bits: head shapes,
lengths around the tile edges, empty and invalid sequences, hostile
neighbours, strided operands, captured calls."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, attend, check_attention, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def views(x, H, Hkv, dq, dv):
    q, k, v = x.split([H * dq, Hkv * dq, Hkv * dv], dim=1)
    return q.unflatten(1, (H, dq)), k.unflatten(1, (Hkv, dq)), v.unflatten(1, (Hkv, dv))


def starts(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32)


def check_sequences(out, lse, q, k, v, cu, dq, scale=None):
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if hi > lo:
            ref = attend(q[lo:hi], k[lo:hi], v[lo:hi], scale or dq ** -0.5, True)
            check_attention(out[lo:hi], None if lse is None else lse[:, lo:hi], ref, dq, HALF_BF16, f"sequence {b} ({hi - lo} tokens)")


LENS = [1, 0, 2, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257, 400]
SHAPES = [
    # H, Hkv, dq, dv
    (8, 2, 128, 128), (4, 4, 128, 128), (16, 1, 128, 128), (6, 2, 64, 64), (5, 1, 64, 128), (14, 2, 128, 64),
    (3, 3, 192, 128), (12, 1, 192, 64), (8, 1, 64, 64), (26, 2, 128, 128), (22, 2, 192, 128), (30, 2, 64, 64), (2, 1, 192, 128),
]


# Up to 128 rows a sequence (rows of none among them) run with one query tile a CTA, more with pairs of tiles.
@pytest.mark.parametrize("times,rest", [(1, 5), (1, 900), (4, 2500)])
@pytest.mark.parametrize("H,Hkv,dq,dv", SHAPES + [(32, 8, 128, 128), (24, 8, 64, 128)])
def test_matches_formula(H, Hkv, dq, dv, times, rest):
    cu = starts(LENS * times)
    T = int(cu[-1]) + rest
    x = randn((T, H * dq + Hkv * (dq + dv)), 1)
    q, k, v = views(x, H, Hkv, dq, dv)
    out = torch.full((T, H, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((H, T), 7.0, device=DEV)
    vpp.vpp_prompt_attn(*views(x.to(DEV), H, Hkv, dq, dv), cu.to(DEV), out=out, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_sequences(out, lse, q, k, v, cu, dq)
    assert bool((out[int(cu[-1]):] == 7).all()) and bool((lse[:, int(cu[-1]):] == 7).all()), "rows of no sequence written"


@pytest.mark.parametrize("lens", [[1], [128], [3, 1500], [1] * 300, [2000], [0, 0, 5, 0], [513, 700, 1, 1, 1025]])
def test_batch_shapes(lens):
    H, Hkv, d = 8, 2, 128
    cu = starts(lens)
    q, k, v = randn((int(cu[-1]), H, d), 2), randn((int(cu[-1]), Hkv, d), 3), randn((int(cu[-1]), Hkv, d), 4)
    lse = torch.empty((H, int(cu[-1])), device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_sequences(out, lse, q, k, v, cu, d)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (6, 2, 64), (2, 2, 128), (32, 8, 128), (48, 16, 64)])
@pytest.mark.parametrize("rest", [9, 1000])
def test_neighbours_never_reach_a_result(H, Hkv, d, bad, rest):
    """Sequences of hostile values before and behind each good one, and in the rows of no sequence."""
    lens = [30, 100, 40, 129, 10, 200, 3]
    cu = starts(lens)
    T = int(cu[-1]) + rest
    q, k, v = randn((T, H, d), 5), randn((T, Hkv, d), 6), randn((T, Hkv, d), 7)
    good = [1, 3, 5]
    for b in range(len(lens)):
        if b not in good:
            for x in (q, k, v):
                x[int(cu[b]):int(cu[b + 1])] = bad
    for x in (q, k, v):
        x[int(cu[-1]):] = bad
    lse = torch.empty((H, T), device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse)
    for b in good:
        lo, hi = int(cu[b]), int(cu[b + 1])
        ref = attend(q[lo:hi], k[lo:hi], v[lo:hi], d ** -0.5, True)
        check_attention(out[lo:hi], lse[:, lo:hi], ref, d, HALF_BF16, f"sequence {b}")


def test_scale_and_no_lse():
    H, Hkv, d = 4, 2, 64
    cu = starts([100, 30])
    q, k, v = randn((130, H, d), 8), randn((130, Hkv, d), 9), randn((130, Hkv, d), 10)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), softmax_scale=0.4)
    check_sequences(out, None, q, k, v, cu, d, scale=0.4)


@pytest.mark.parametrize("T", [100, 600])
def test_invalid_ranges_are_left_out_and_reported(T):
    H, Hkv, d = 4, 2, 64
    q, k, v = randn((T, H, d), 11), randn((T, Hkv, d), 12), randn((T, Hkv, d), 13)
    for cu in ([0, 40, 30, T], [0, 40, 60, T + 100], [-20, 10, 50, T], [0, 40, 1 << 30, T]):
        out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), out=out)
        assert vpp.vpp_last_device_status() == vpp.VPP_ERR_INVALID, cu
        rest = torch.ones(T, dtype=torch.bool)
        for lo, hi in zip(cu, cu[1:]):
            if 0 <= lo <= hi <= T:
                rest[lo:hi] = False
        assert bool((out.cpu()[rest] == 7).all()), cu
    # a valid sequence beside the invalid ones is served
    cu = [0, 40, 60, T + 100]
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV))
    check_sequences(out, None, q, k, v, cu[:3], d)
    assert vpp.vpp_last_device_status() == vpp.VPP_ERR_INVALID


def test_equals_the_cached_path():
    """A whole prompt through the paged cache and through the packed call: the same attention."""
    H, Hkv, d, n = 16, 4, 128, 700
    q, k, v = (randn((n, h, d), 14 + h).to(DEV) for h in (H, Hkv, Hkv))
    cu = torch.tensor([0, n], dtype=torch.int32)
    table = torch.arange((n + 63) // 64, dtype=torch.int32, device=DEV)[None]
    kc = torch.zeros((table.shape[1], 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    vpp.vpp_kv_append_varlen(k, v, kc, vc, table, cu.numpy(), [n])
    a = vpp.vpp_mixed_attn(q, kc, vc, table, cu.numpy(), [n])
    b = vpp.vpp_prompt_attn(q, k, v, cu.to(DEV))
    check_sequences(b, None, q.cpu(), k.cpu(), v.cpu(), cu, d)
    check_sequences(a, None, q.cpu(), k.cpu(), v.cpu(), cu, d)


def test_runs_give_the_same_bits():
    H, Hkv, d = 8, 2, 128
    lens = [300, 1, 77, 512, 0, 64]
    cu = starts(lens)
    T = int(cu[-1])
    q, k, v = randn((T, H, d), 15).to(DEV), randn((T, Hkv, d), 16).to(DEV), randn((T, Hkv, d), 17).to(DEV)
    want = vpp.vpp_prompt_attn(q, k, v, cu.to(DEV))
    for _ in range(5):
        assert torch.equal(vpp.vpp_prompt_attn(q, k, v, cu.to(DEV)), want)


def test_captured_call_follows_the_lengths():
    H, Hkv, d, T = 8, 2, 128, 900
    q, k, v = randn((T, H, d), 18), randn((T, Hkv, d), 19), randn((T, Hkv, d), 20)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    cu = torch.zeros(7, dtype=torch.int32, device=DEV)
    out, lse = torch.empty((T, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((H, T), device=DEV)
    vpp.vpp_prompt_attn(qd, kd, vd, cu, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vpp.vpp_prompt_attn(qd, kd, vd, cu, out=out, lse=lse)
    for lens in ([900, 0, 0, 0, 0, 0], [100] * 6, [1, 2, 3, 4, 5, 6], [0, 0, 0, 0, 0, 900], [450, 300, 50, 60, 39, 1]):
        now = starts(lens)
        cu.copy_(now)
        out.fill_(7.0)
        graph.replay()
        check_sequences(out, lse, q, k, v, now, d)
        assert bool((out[int(now[-1]):] == 7).all())
    assert vpp.vpp_last_device_status() == 0


def test_another_stream():
    H, Hkv, d = 8, 2, 128
    cu = starts([500, 30, 200])
    q, k, v = (randn((730, h, d), 21 + h).to(DEV) for h in (H, Hkv, Hkv))
    want = vpp.vpp_prompt_attn(q, k, v, cu.to(DEV))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    cud = cu.to(DEV)
    torch.cuda.synchronize()
    got = [vpp.vpp_prompt_attn(q, k, v, cud, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


@pytest.mark.parametrize("n,power", [(900, 6), (300, 2)])
def test_many_ragged_sequences(n, power):
    """More sequences than the work list keeps in registers, of very different lengths, empty ones among them."""
    H, Hkv, d = 8, 4, 64
    g = torch.Generator().manual_seed(30)
    lens = [int(x) for x in (torch.rand(n, generator=g) ** power * 500).long()]
    lens[17], lens[n // 3 * 2], lens[n - 1] = 900, 0, 333
    cu = starts(lens)
    T = int(cu[-1])
    q, k, v = randn((T, H, d), 31), randn((T, Hkv, d), 32), randn((T, Hkv, d), 33)
    lse = torch.full((H, T), 7.0, device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_sequences(out, lse, q, k, v, cu, d)


@pytest.mark.parametrize("H,Hkv,d", [(8, 8, 128), (32, 8, 64)])
@pytest.mark.parametrize("empty", [0, 300])
def test_few_live_rows_of_many(H, Hkv, d, empty):
    """A launch sized for many rows of which almost none belong to a sequence."""
    T = 20000
    q, k, v = (torch.full((T, h, d), float("nan"), dtype=torch.bfloat16, device=DEV) for h in (H, Hkv, Hkv))
    live = [randn((70, h, d), 34 + h) for h in (H, Hkv, Hkv)]
    for x, y in zip((q, k, v), live):
        x[5:75] = y.to(DEV)
    cu = torch.tensor([5, 5, 75, 75] + [75] * empty, dtype=torch.int32)
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vpp.vpp_prompt_attn(q, k, v, cu.to(DEV), out=out)
    check_sequences(out[5:75], None, *live, [0, 70], d)
    assert bool((out[:5] == 7).all()) and bool((out[75:] == 7).all())
    assert vpp.vpp_last_device_status() == 0


def test_growing_scores_rescale():
    """Keys whose scores grow along a long sequence, so that the running maximum moves on nearly every tile."""
    H, Hkv, d, n = 32, 8, 128, 1300
    base = randn((H, d), 40).float()
    ramp = torch.linspace(0.2, 3, n)
    q = base[None].expand(n, H, d).to(torch.bfloat16)
    k = (ramp[:, None, None] * base[:: H // Hkv][None]).to(torch.bfloat16)
    v = randn((n, Hkv, d), 41)
    cu = starts([n])
    lse = torch.empty((H, n), device=DEV)
    out = vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), lse=lse, softmax_scale=0.2)
    check_sequences(out, lse, q, k, v, cu, d, scale=0.2)


@pytest.mark.parametrize("Hkv,lens", [(40, [300, 10500, 7]), (64, [6500, 2])])
def test_heads_in_groups(Hkv, lens):
    """Keys and values of all heads beyond 100 MB (the items then go by groups of heads, the last group a partial one):
    sampled rows against the formula, and every row written once or more."""
    d = 64
    cu = starts(lens)
    T = int(cu[-1])
    q, k, v = randn((T, Hkv, d), 31), randn((T, Hkv, d), 32), randn((T, Hkv, d), 33)
    out = torch.full((T, Hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Hkv, T), float("nan"), device=DEV)
    vpp.vpp_prompt_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), out=out, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for b, n in enumerate(lens):
        lo = int(cu[b])
        for t in sorted({0, n // 3, n // 2 + 1, n - 1}):
            ref = attend(q[lo + t:lo + t + 1], k[lo:lo + t + 1], v[lo:lo + t + 1], d ** -0.5, False)
            # (besides P's rounding, t + 1 products added up in float32)
            check_attention(out[lo + t:lo + t + 1], lse[:, lo + t:lo + t + 1], ref, d, HALF_BF16 + (t + 1) * 2.0 ** -23,
                            f"sequence {b} token {t}")


@pytest.mark.parametrize("H,Hkv,dq,dv", [(64, 8, 128, 128), (64, 4, 192, 128)])
def test_offsets_past_32_bits(H, Hkv, dq, dv):
    """A sequence at the far end of more than 2^31 elements of queries and of output."""
    n, T = 300, (1 << 31) // (H * 128) + 400
    q = torch.zeros((T, H, dq), dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device=DEV) for d in (dq, dv))
    live = randn((n, H, dq), 50), randn((n, Hkv, dq), 51), randn((n, Hkv, dv), 52)
    for x, y in zip((q, k, v), live):
        x[T - n:] = y.to(DEV)
    cu = torch.tensor([T - n, T], dtype=torch.int32, device=DEV)
    out = torch.zeros((T, H, dv), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((H, T), device=DEV)
    vpp.vpp_prompt_attn(q, k, v, cu, out=out, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_sequences(out[T - n:], lse[:, T - n:], *live, [0, n], dq)
    assert not bool(out[:T - n].any()) and not bool(lse[:, :T - n].any())
