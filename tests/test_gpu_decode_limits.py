"""Decode attention with device lengths at the ends of its ranges, beside the host-planned call, and over shared blocks."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, HALF_F16, attend, check_attention, randn
from tests.test_gpu_decode_paged import call, check_rows, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv", [(1024, 1024), (2048, 1024), (3900, 300), (610, 610)])
def test_many_kv_heads(H, Hkv, fp8):
    """Up to 1024 kv heads: one column of pages, where no sequence is ever split."""
    ctx, d = [1, 130, 0, 64], 64
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, fp8)
    q = randn((len(ctx), H, d), 3)
    lse = torch.full((H, len(ctx)), 3.0, device=DEV)
    out = call(fp8, q.to(DEV), kc, vc, ks, vs, table, ctx, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_rows(out, lse, q, keys, vals, ctx, d, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_sequences_may_share_blocks(fp8):
    """A common prefix held once: the same blocks in several rows, and the same block twice in one row."""
    H, Hkv, d = 8, 2, 128
    kc, vc, ks, vs, table, keys, vals = make([300], Hkv, d, d, fp8)
    shared = table[0].expand(4, -1).clone()
    shared[3, 1] = shared[3, 0]
    ctx = [300, 130, 1, 128]
    q = randn((4, H, d), 4)
    twice = [torch.cat([x[0][:64], x[0][:64]]) for x in (keys, vals)]
    lse = torch.empty((H, 4), device=DEV)
    out = call(fp8, q.to(DEV), kc, vc, ks, vs, shared, ctx, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    rows = [(keys[0][:n], vals[0][:n]) for n in ctx[:3]] + [tuple(twice)]
    check_rows(out, lse, q, [k for k, _ in rows], [v for _, v in rows], ctx, d, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_host_planned_call_gives_the_same_rows(fp8):
    """Decode rows of vpp_mixed_attn and the device-planned call: within both tolerances of each other."""
    H, Hkv, d = 16, 4, 128
    ctx = [900, 1, 64, 2500]
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, fp8, dead=0.0)
    q = randn((4, H, d), 5)
    cu = list(range(5))
    if fp8:
        a = vpp.vpp_mixed_attn_fp8(q.to(DEV), kc, vc, ks, vs, table, cu, ctx)
    else:
        a = vpp.vpp_mixed_attn(q.to(DEV), kc, vc, table, cu, ctx)
    lse = torch.empty((H, 4), device=DEV)
    b = call(fp8, q.to(DEV), kc, vc, ks, vs, table, ctx, lse=lse)
    half = HALF_F16 if fp8 else HALF_BF16
    for i in range(4):
        ref = attend(q[i:i + 1], keys[i], vals[i], d ** -0.5, False)
        check_attention(b[i:i + 1], lse[:, i:i + 1], ref, d, half, f"row {i}")
        o, _, absw, _ = ref
        # each side: P to its operand type (bf16 at most), one rounding to bf16 (2^-14 holds check_attention's float32 terms)
        tol = 2 * (HALF_BF16 * o.abs() + (HALF_BF16 + 2.0 ** -14) * absw)
        assert bool(((a[i:i + 1].double().cpu() - b[i:i + 1].double().cpu()).abs() <= tol).all())


def test_ten_thousand_rows():
    """More rows than a warp scans at once, almost all of length 0 or 1."""
    H, Hkv, d = 2, 1, 64
    ctx = [0] * 10000
    for i in range(7, 10000, 331):
        ctx[i] = 1 + (i * 7) % 190
    kc, vc, ks, vs, table, keys, vals = make(ctx, Hkv, d, d, False)
    q = randn((len(ctx), H, d), 6)
    lse = torch.full((H, len(ctx)), 3.0, device=DEV)
    out = call(False, q.to(DEV), kc, vc, ks, vs, table, ctx, lse=lse)
    assert vpp.vpp_last_device_status() == 0
    check_rows(out, lse, q, keys, vals, ctx, d, False)
