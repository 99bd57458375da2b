"""Decode attention with device lengths against the formula in 64 bits: every
head shape, lengths around the block edges, padding rows, hostile values in
dead cache rows, E4M3 caches, strided queries, reused workspaces."""

import math

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, HALF_F16, attend, block_table, check_attention, fill_cache, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(ctx, Hkv, dq, dv, fp8, seed=0, dead=float("nan"), spare=2):
    """Caches whose dead rows hold `dead`, the table, and each row's k and v (as stored values)."""
    table, pool = block_table(ctx, seed, spare)
    kc, vc = (torch.full((pool, 64, Hkv, d), dead, dtype=torch.float32).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
              for d in (dq, dv))
    if fp8:
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    ks = 0.02 + 0.02 * torch.rand(Hkv, generator=torch.Generator().manual_seed(seed))
    vs = 0.02 + 0.02 * torch.rand(Hkv, generator=torch.Generator().manual_seed(seed + 1))
    keys, vals = [], []
    for b, n in enumerate(ctx):
        k, v = randn((n, Hkv, dq), 100 + seed + b), randn((n, Hkv, dv), 900 + seed + b)
        if fp8:
            k8 = (k.float() / ks[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            v8 = (v.float() / vs[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            fill_cache(kc, table, b, k8.view(torch.uint8))
            fill_cache(vc, table, b, v8.view(torch.uint8))
            k, v = k8.double() * ks.double()[:, None], v8.double() * vs.double()[:, None]
        else:
            fill_cache(kc, table, b, k)
            fill_cache(vc, table, b, v)
        keys.append(k)
        vals.append(v)
    return kc.to(DEV), vc.to(DEV), ks.to(DEV), vs.to(DEV), table.to(DEV), keys, vals


def call(fp8, q, kc, vc, ks, vs, table, ctx, **kw):
    c = ctx if torch.is_tensor(ctx) else torch.tensor(ctx, dtype=torch.int32, device=DEV)
    if fp8:
        return vpp.vpp_decode_attn_fp8(q, kc, vc, ks, vs, table, c, **kw)
    return vpp.vpp_decode_attn(q, kc, vc, table, c, **kw)


def check_rows(out, lse, q, keys, vals, ctx, dq, fp8, scale=None):
    for b, n in enumerate(ctx):
        if n == 0:
            assert not bool(out[b].any()), f"row {b} is empty"
            assert bool((lse[:, b] == -math.inf).all())
            continue
        ref = attend(q[b:b + 1], keys[b], vals[b], scale or dq ** -0.5, False)
        check_attention(out[b:b + 1], lse[:, b:b + 1], ref, dq, HALF_F16 if fp8 else HALF_BF16, f"row {b}, {n} keys")


CTX = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700, 0, 1500, 2048]
SHAPES = [
    # H, Hkv, dq, dv
    (32, 8, 128, 128), (8, 8, 128, 128), (16, 1, 128, 128), (9, 3, 64, 64), (12, 12, 64, 128), (10, 2, 128, 64),
    (16, 16, 192, 128), (14, 2, 192, 64), (7, 1, 64, 64), (64, 8, 128, 128), (48, 4, 128, 128), (40, 40, 192, 128),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv,dq,dv", SHAPES)
def test_matches_formula(H, Hkv, dq, dv, fp8):
    kc, vc, ks, vs, table, keys, vals = make(CTX, Hkv, dq, dv, fp8)
    q = randn((len(CTX), H, dq), 5)
    lse = torch.full((H, len(CTX)), 3.0, device=DEV)
    out = call(fp8, q.to(DEV), kc, vc, ks, vs, table, CTX, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_rows(out, lse, q, keys, vals, CTX, dq, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx", [[1], [64], [65], [9000], [0], [0, 0, 0], [40000, 1, 0, 3], [1] * 400, [0] * 50 + [5000] + [0] * 50 + [77]])
def test_batch_shapes(ctx, fp8):
    """One row, all padding, one long row among short ones, many one-token rows, long runs of padding."""
    H, Hkv, d = 8, 2, 128
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, fp8)
    q = randn((len(ctx), H, d), 6)
    lse = torch.full((H, len(ctx)), 3.0, device=DEV)
    out = call(fp8, q.to(DEV), kc, vc, ks, vs, table, ctx, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_rows(out, lse, q, keys, vals, ctx, d, fp8)


@pytest.mark.parametrize("dead", [float("inf"), -float("inf"), 3.0e38])
def test_dead_cache_rows_may_hold_anything(dead):
    ctx = [1, 33, 64, 100]
    kc, vc, ks, vs, table, keys, vals = make(ctx, 2, 128, 128, False, dead=dead)
    q = randn((len(ctx), 8, 128), 7)
    lse = torch.empty((8, len(ctx)), device=DEV)
    out = call(False, q.to(DEV), kc, vc, ks, vs, table, ctx, lse=lse)
    check_rows(out, lse, q, keys, vals, ctx, 128, False)


@pytest.mark.parametrize("fp8", [False, True])
def test_strided_queries_scale_no_lse(fp8):
    H, Hkv, d = 12, 4, 64
    ctx = [5, 300, 64, 0]
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, fp8)
    wide = randn((len(ctx), (H + 2 * Hkv) * d), 8)
    q = wide[:, : H * d].unflatten(1, (H, d))
    qd = wide.to(DEV)[:, : H * d].unflatten(1, (H, d))
    out = torch.full((len(ctx), H, d), 9.0, dtype=torch.bfloat16, device=DEV)
    ret = call(fp8, qd, kc, vc, ks, vs, table, ctx, out=out, softmax_scale=0.3)
    assert ret is out
    lse = torch.empty((H, len(ctx)), device=DEV)
    call(fp8, qd, kc, vc, ks, vs, table, ctx, lse=lse, softmax_scale=0.3)
    check_rows(out, lse, q, keys, vals, ctx, d, fp8, scale=0.3)


@pytest.mark.parametrize("fp8", [False, True])
def test_growing_scores_rescale(fp8):
    """Keys whose scores grow along the sequence, so that the running maximum moves on nearly every tile, and rows of
    equal keys; the largest score is at the end, in the middle and at the start."""
    H, Hkv, d, n = 4, 2, 128, 1400
    ctx = [n, n, n, n]
    kc, vc, ks, vs, table, _, vals = make(ctx, Hkv, d, d, fp8)
    q = randn((4, H, d), 9)
    base = q.float()[:, :: H // Hkv].mean(0)  # one direction per kv head
    keys = []
    host = kc.cpu()
    for b, shape in enumerate(("up", "peak", "down", "flat")):
        ramp = {"up": torch.linspace(-3, 3, n), "down": torch.linspace(3, -3, n), "flat": torch.ones(n),
                "peak": 3 - (torch.linspace(-2, 2, n) ** 2)}[shape]
        k = (ramp[:, None, None] * base[None]).to(torch.bfloat16)
        if fp8:
            k8 = (k.float() / ks.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            fill_cache(host, table.cpu(), b, k8.view(torch.uint8))
            keys.append(k8.double() * ks.cpu().double()[:, None])
        else:
            fill_cache(host, table.cpu(), b, k)
            keys.append(k)
    lse = torch.empty((H, 4), device=DEV)
    out = call(fp8, q.to(DEV), host.to(DEV), vc, ks, vs, table, ctx, lse=lse, softmax_scale=0.5)
    check_rows(out, lse, q, keys, vals, ctx, d, fp8, scale=0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_blocks(fp8):
    """A length outside the table's row empties the row, a block outside the pool reads as zeros; both are reported."""
    H, Hkv, d = 4, 2, 64
    ctx = [70, 100, 10, 128]
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, fp8)
    q = randn((4, H, d), 11)
    table[3, 0] = 1 << 20
    keys[3], vals[3] = keys[3].clone(), vals[3].clone()
    keys[3][:64], vals[3][:64] = 0, 0
    lens = torch.tensor([70, -1, 129, 128], dtype=torch.int32, device=DEV)
    lse = torch.empty((H, 4), device=DEV)
    out = call(fp8, q.to(DEV), kc, vc, ks, vs, table, lens, lse=lse)
    assert vpp.vpp_last_device_status() == vpp.VPP_ERR_INVALID
    check_rows(out, lse, q, keys, vals, [70, 0, 0, 128], d, fp8)
    assert vpp.vpp_last_device_status() == 0


def test_runs_give_the_same_bits_and_a_dirty_workspace_is_fine():
    H, Hkv, d = 32, 8, 128
    ctx = [3000, 17, 0, 12345, 640]
    kc, vc, ks, vs, table, _, _ = make(ctx, Hkv, d, d, False)
    q = randn((len(ctx), H, d), 12).to(DEV)
    size = vpp.decode_attn_workspace_size(len(ctx), H, Hkv, d, d)
    ws = torch.full((max(size, 16),), 255, dtype=torch.uint8, device=DEV)
    lse = torch.empty((H, len(ctx)), device=DEV)
    first = call(False, q, kc, vc, ks, vs, table, ctx, lse=lse, workspace=ws).clone()
    first_lse = lse.clone()
    for fill in (0, 127, 255):
        ws.fill_(fill)
        out = call(False, q, kc, vc, ks, vs, table, ctx, lse=lse, workspace=ws)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


def test_a_small_workspace_is_refused():
    H, Hkv, d = 32, 8, 128
    size = vpp.decode_attn_workspace_size(4, H, Hkv, d, d)
    kc, vc, ks, vs, table, _, _ = make([100] * 4, Hkv, d, d, False)
    q = randn((4, H, d), 13).to(DEV)
    if size > 0:
        with pytest.raises(vpp.VppError) as e:
            call(False, q, kc, vc, ks, vs, table, [100] * 4, workspace=torch.empty(size - 1, dtype=torch.uint8, device=DEV))
        assert e.value.code == vpp.VPP_ERR_WORKSPACE


def test_captured_call_follows_the_lengths():
    """One captured call replayed with other lengths, tables and queries equals eager calls, bit for bit."""
    H, Hkv, d = 16, 4, 128
    most = [5000, 200, 64, 1, 900]
    kc, vc, ks, vs, table, keys, vals = make(most, Hkv, d, d, False)
    q = randn((5, H, d), 14).to(DEV)
    lens = torch.zeros(5, dtype=torch.int32, device=DEV)
    out, lse = torch.empty((5, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((H, 5), device=DEV)
    ws = torch.empty(vpp.decode_attn_workspace_size(5, H, Hkv, d, d) + 16, dtype=torch.uint8, device=DEV)
    call(False, q, kc, vc, ks, vs, table, lens, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(False, q, kc, vc, ks, vs, table, lens, out=out, lse=lse, workspace=ws)
    for now in ([1, 1, 1, 1, 1], [5000, 0, 64, 1, 0], [4999, 200, 3, 0, 900], [0] * 5, [64, 128, 0, 1, 65]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        a, al = out.clone(), lse.clone()
        el = torch.empty_like(lse)
        e = call(False, q, kc, vc, ks, vs, table, now, lse=el)
        assert torch.equal(a, e) and torch.equal(al, el)
        check_rows(a, al, q.cpu(), [k[:n] for k, n in zip(keys, now)], [v[:n] for v, n in zip(vals, now)], now, d, False)
    assert vpp.vpp_last_device_status() == 0


def test_two_streams_with_their_own_workspaces():
    H, Hkv, d = 16, 4, 128
    ctx = [3000, 50, 700]
    kc, vc, ks, vs, table, _, _ = make(ctx, Hkv, d, d, False)
    qs = [randn((3, H, d), 20 + i).to(DEV) for i in range(2)]
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    want = [call(False, q, kc, vc, ks, vs, table, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(call(False, qs[i], kc, vc, ks, vs, table, lens, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_offsets_past_32_bits():
    """Blocks at the far end of a pool of more than 2^32 elements a cache."""
    H, Hkv, d = 8, 8, 128
    pool = (1 << 32) // (64 * Hkv * d) + 40
    kc = torch.zeros((pool, 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    ctx = [150, 64]
    table = torch.tensor([[pool - 1, 0, pool - 7], [pool - 3, -1, -1]], dtype=torch.int32)
    keys, vals = [], []
    for b, n in enumerate(ctx):
        k, v = randn((n, Hkv, d), 30 + b), randn((n, Hkv, d), 40 + b)
        for i in range(0, n, 64):
            m = min(64, n - i)
            kc[int(table[b, i // 64]), :m] = k[i:i + m].to(DEV)
            vc[int(table[b, i // 64]), :m] = v[i:i + m].to(DEV)
        keys.append(k)
        vals.append(v)
    q = randn((2, H, d), 50)
    lse = torch.empty((H, 2), device=DEV)
    out = call(False, q.to(DEV), kc, vc, None, None, table.to(DEV), ctx, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_rows(out, lse, q, keys, vals, ctx, d, False)


def test_captured_and_eager_calls_without_a_workspace_do_not_share_one():
    """A captured call that was given no workspace is replayed on one stream while eager calls run on another and on the
    stream of the capture."""
    H, Hkv, d = 16, 4, 128
    ctx = [4000, 50, 1700]
    kc, vc, ks, vs, table, _, _ = make(ctx, Hkv, d, d, False)
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    qa, qb = randn((3, H, d), 60).to(DEV), randn((3, H, d), 61).to(DEV)
    want_a, want_b = call(False, qa, kc, vc, ks, vs, table, lens), call(False, qb, kc, vc, ks, vs, table, lens)
    out = torch.empty_like(want_a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(False, qa, kc, vc, ks, vs, table, lens, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(30):
        with torch.cuda.stream(side):
            graph.replay()
        got.append(call(False, qb, kc, vc, ks, vs, table, lens))
    torch.cuda.synchronize()
    assert torch.equal(out, want_a)
    assert all(torch.equal(o, want_b) for o in got)


def test_threads_on_one_stream():
    """Several host threads call on the same stream: a call is two launches, and each thread has its own workspace."""
    import threading

    H, Hkv, d = 16, 4, 128
    ctx = [4000, 50, 1700]
    kc, vc, ks, vs, table, _, _ = make(ctx, Hkv, d, d, False)
    lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    qs = [randn((3, H, d), 70 + i).to(DEV) for i in range(4)]
    want = [call(False, q, kc, vc, ks, vs, table, lens) for q in qs]
    got = [[] for _ in qs]

    def work(i):
        for _ in range(50):
            got[i].append(call(False, qs[i], kc, vc, ks, vs, table, lens))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_infinite_scores():
    """A row whose scores are all -inf has weights that sum to nothing (0 and -inf, as an empty row); a NaN key gives NaN
    to the heads that read it and to no other row."""
    H, Hkv, d = 4, 2, 64
    ctx = [40, 40, 40]
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, False)
    q = torch.ones((3, H, d), dtype=torch.bfloat16)
    host = kc.cpu()
    keys[0][:, 0] = float("-inf")
    keys[1][7, 1] = float("nan")
    for b in (0, 1):
        fill_cache(host, table.cpu(), b, keys[b])
    lse = torch.empty((H, 3), device=DEV)
    out = call(False, q.to(DEV), host.to(DEV), vc, ks, vs, table, ctx, lse=lse).float().cpu()
    assert not bool(out[0, :2].any()) and bool((lse[:2, 0] == -math.inf).all())
    assert bool(out[1, 2:].isnan().all()) and bool(lse[2:, 1].isnan().all())
    assert bool(out[0, 2:].isfinite().all()) and bool(out[1, :2].isfinite().all()) and bool(out[2].isfinite().all())
