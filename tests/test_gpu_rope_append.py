"""Rotate-and-append against the formula in 64 bits: head shapes, pairings,
partial rotations, ragged and padded batches, strided and in-place operands,
E4M3 caches, and what it must leave untouched."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, HALF_E4M3, block_table, randn, rotate, rotate_slack

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cos_sin_table(rows, rot, seed=0):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv[None] + 0.1 * seed
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def make(new, past, H, Hkv, dq, dv, fp8, pad=0, seed=0):
    """A ragged batch on the CPU: fused projection, lengths, table, caches of a known fill."""
    T = sum(new) + pad
    x = randn((T, H * dq + Hkv * (dq + dv)), 10 + seed)
    ctx = [a + b if a else 0 for a, b in zip(new, past)]
    table, pool = block_table(ctx, 3 + seed)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    if fp8:
        kc = torch.randint(0, 120, (pool, 64, Hkv, dq), dtype=torch.uint8)
        vc = torch.randint(0, 120, (pool, 64, Hkv, dv), dtype=torch.uint8)
    else:
        kc, vc = randn((pool, 64, Hkv, dq), 20), randn((pool, 64, Hkv, dv), 21)
    return x, cu, torch.tensor(ctx, dtype=torch.int32), table, kc, vc


def views(x, H, Hkv, dq, dv):
    q, k, v = x.split([H * dq, Hkv * dq, Hkv * dv], dim=1)
    return q.unflatten(1, (H, dq)), k.unflatten(1, (Hkv, dq)), v.unflatten(1, (Hkv, dv))


def slots(cu, ctx, table):
    """(token, position, block, row) of every live token."""
    t, pos, blk = [], [], []
    for b in range(len(ctx)):
        lo, hi, c = int(cu[b]), int(cu[b + 1]), int(ctx[b])
        for i in range(lo, hi):
            if c:
                p = c - (hi - i)
                t.append(i), pos.append(p), blk.append(int(table[b, p // 64]))
    return torch.tensor(t), torch.tensor(pos), torch.tensor(blk), torch.tensor(pos) % 64


def check_bf16(got, ref, slack, what):
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= HALF_BF16 * ref.abs() + slack * 1.01).all()), f"{what}: {float(err.max())}"


SHAPES = [
    # H, Hkv, dq, dv, rot, start, interleaved
    (8, 2, 128, 128, 128, 0, False),
    (8, 2, 128, 128, 128, 0, True),
    (4, 4, 64, 64, 64, 0, False),
    (6, 1, 64, 128, 32, 0, True),
    (5, 5, 192, 128, 64, 128, True),
    (3, 1, 192, 64, 48, 96, False),
    (14, 2, 128, 64, 16, 8, False),
    (2, 1, 128, 128, 0, 0, False),
    (64, 8, 128, 128, 128, 0, False),
    (2, 2, 256, 64, 256, 0, False),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv,dq,dv,rot,start,il", SHAPES)
def test_matches_formula(H, Hkv, dq, dv, rot, start, il, fp8):
    new = [1, 0, 63, 64, 2, 130, 1, 5]
    past = [0, 9, 1, 0, 126, 3, 1000, 61]
    x, cu, ctx, table, kc, vc = make(new, past, H, Hkv, dq, dv, fp8, pad=3)
    q, k, v = views(x, H, Hkv, dq, dv)
    cs = cos_sin_table(1001, rot) if rot else None
    ks = 0.01 + 0.02 * torch.rand(Hkv, generator=torch.Generator().manual_seed(1))
    vs = 0.01 + 0.02 * torch.rand(Hkv, generator=torch.Generator().manual_seed(2))
    xd = x.to(DEV)
    qd, kd, vd = views(xd, H, Hkv, dq, dv)
    kcd, vcd = kc.to(DEV), vc.to(DEV)
    qo = torch.full((x.shape[0], H, dq), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((x.shape[0], Hkv, dq), 7.0, dtype=torch.bfloat16, device=DEV)
    args = (table.to(DEV), cu.to(DEV), ctx.to(DEV))
    kw = dict(q_out=qo, k_out=ko, rot_start=start, interleaved=il)
    csd = None if cs is None else cs.to(DEV)
    if fp8:
        vpp.vpp_rope_append_fp8(qd, kd, vd, csd, kcd, vcd, ks.to(DEV), vs.to(DEV), *args, **kw)
    else:
        vpp.vpp_rope_append(qd, kd, vd, csd, kcd, vcd, *args, **kw)
    assert vpp.vpp_last_device_status() == 0
    assert torch.equal(xd.cpu(), x), "inputs changed"
    t, pos, blk, row = slots(cu, ctx, table)
    slack = rotate_slack(x, cs)
    rq, rk = rotate(q[t], pos, cs, start, il), rotate(k[t], pos, cs, start, il)
    check_bf16(qo[t.to(DEV)], rq, slack, "q_out")
    check_bf16(ko[t.to(DEV)], rk, slack, "k_out")
    dead = torch.ones(x.shape[0], dtype=torch.bool)
    dead[t] = False
    assert bool((qo.cpu()[dead] == 7).all()) and bool((ko.cpu()[dead] == 7).all()), "padding rows written"
    for cache, got, ref, scale, sl in ((kc, kcd.cpu(), rk, ks, slack), (vc, vcd.cpu(), v[t].double(), vs, 0.0)):
        if fp8:
            want = (ref / scale.double()[:, None]).clamp(-448, 448)
            have = got[blk, row].view(torch.float8_e4m3fn).double()
            # half a step (2^-10 below the normal range), and the float32 rotation and quotient before it
            tol = torch.clamp(HALF_E4M3 * want.abs(), min=2.0 ** -10) + 1.1 * sl / scale.double()[:, None] + 2.0 ** -23 * want.abs()
            assert bool(((have - want).abs() <= tol).all())
        else:
            check_bf16(got[blk, row], ref, sl, "cache")
        rest = torch.ones(cache.shape[:2], dtype=torch.bool)
        rest[blk, row] = False
        assert torch.equal(got[rest], cache[rest]), "other cache rows changed"


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("rot,start", [(128, 0), (64, 32)])
def test_in_place_equals_out_of_place(rot, start, il):
    H, Hkv, d = 8, 2, 128
    new, past = [5, 70, 1], [0, 10, 300]
    x, cu, ctx, table, kc, vc = make(new, past, H, Hkv, d, d, False, pad=2)
    cs = cos_sin_table(512, rot).to(DEV)
    args = (table.to(DEV), cu.to(DEV), ctx.to(DEV))
    a, b = x.to(DEV), x.to(DEV)
    qa, ka, va = views(a, H, Hkv, d, d)
    qb, kb, vb = views(b, H, Hkv, d, d)
    c1, c2 = (kc.to(DEV), vc.to(DEV)), (kc.to(DEV), vc.to(DEV))
    qo, ko = qa.contiguous(), ka.contiguous()
    vpp.vpp_rope_append(qa, ka, va, cs, *c1, *args, q_out=qo, k_out=ko, rot_start=start, interleaved=il)
    vpp.vpp_rope_append(qb, kb, vb, cs, *c2, *args, q_out=qb, k_out=kb, rot_start=start, interleaved=il)
    assert torch.equal(qo, qb) and torch.equal(ko, kb) and torch.equal(vb, va)
    assert torch.equal(c1[0], c2[0]) and torch.equal(c1[1], c2[1])
    # keys only, and rotation without a cache, give the same keys and queries
    c3, ko3 = (kc.to(DEV), vc.to(DEV)), ka.contiguous()
    vpp.vpp_rope_append(None, ka, va, cs, *c3, *args, k_out=ko3, rot_start=start, interleaved=il)
    assert torch.equal(ko3, ko) and torch.equal(c3[0], c1[0]) and torch.equal(c3[1], c1[1])
    qo4, ko4 = qa.contiguous(), ka.contiguous()
    vpp.vpp_rope_append(qa, ka, None, cs, None, None, None, args[1], args[2], q_out=qo4, k_out=ko4, rot_start=start, interleaved=il)
    assert torch.equal(qo4, qo) and torch.equal(ko4, ko)
    assert vpp.vpp_last_device_status() == 0


def test_whole_prompts_without_ctx_lens():
    H, Hkv, d = 4, 2, 64
    new = [70, 3, 128]
    x, cu, ctx, table, kc, vc = make(new, [0, 0, 0], H, Hkv, d, d, False)
    cs = cos_sin_table(128, d).to(DEV)
    q, k, v = views(x.to(DEV), H, Hkv, d, d)
    got = []
    for c in (None, ctx.to(DEV)):
        caches = kc.to(DEV), vc.to(DEV)
        got.append((vpp.vpp_rope_append(q, k, v, cs, *caches, table.to(DEV), cu.to(DEV), c), *caches))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_bf16_append_equals_the_plain_append():
    """Without a rotation the caches are bit for bit those of vpp_kv_append_varlen."""
    Hkv, d = 4, 128
    new, past = [1, 64, 33], [64, 0, 100]
    x, cu, ctx, table, kc, vc = make(new, past, 4, Hkv, d, d, False)
    _, k, v = views(x.to(DEV), 4, Hkv, d, d)
    a, b = (kc.to(DEV), vc.to(DEV)), (kc.to(DEV), vc.to(DEV))
    vpp.vpp_rope_append(None, k, v, None, *a, table.to(DEV), cu.to(DEV), ctx.to(DEV))
    vpp.vpp_kv_append_varlen(k.contiguous(), v.contiguous(), *b, table.to(DEV), cu.numpy(), ctx.numpy())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_blocks_are_left_out_and_reported(fp8):
    """Checked in the kernel before any access: nothing is written for such tokens, the others are served."""
    H, Hkv, d = 4, 2, 64
    new, past = [2, 3, 1, 4, 2, 2], [0, 10, 200, 0, 0, 126]
    x, cu, ctx, table, kc, vc = make(new, past, H, Hkv, d, d, fp8)
    ctx[1] = 2          # fewer positions than new tokens
    ctx[2] = 100000     # outside the block table's row (and the cos / sin table)
    table[3, 0] = 4000  # outside the pool
    table[4, 0] = -5
    ctx[5] = 129        # position 128 is behind the cos / sin table, and table entry 2 is unset or absent
    cs = cos_sin_table(128, d).to(DEV)
    q, k, v = views(x.to(DEV), H, Hkv, d, d)
    one = torch.ones(Hkv, device=DEV)
    kcd, vcd = kc.to(DEV), vc.to(DEV)
    qo = torch.full((x.shape[0], H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    args = (table.to(DEV), cu.to(DEV), ctx.to(DEV))
    if fp8:
        vpp.vpp_rope_append_fp8(q, k, v, cs, kcd, vcd, one, one, *args, q_out=qo)
    else:
        vpp.vpp_rope_append(q, k, v, cs, kcd, vcd, *args, q_out=qo)
    assert vpp.vpp_last_device_status() == vpp.VPP_ERR_INVALID
    live = [0, 1, 12]  # sequence 0, and position 127 of sequence 5
    rest = [i for i in range(x.shape[0]) if i not in live]
    assert bool((qo[rest] == 7).all())
    pos = torch.tensor([0, 1, 127])
    check_bf16(qo[live], rotate(views(x, H, Hkv, d, d)[0][live], pos, cs.cpu(), 0, False), rotate_slack(x, cs), "q_out")
    rows = torch.ones(kc.shape[:2], dtype=torch.bool)
    rows[table[0, 0], 0:2] = False
    rows[table[5, 1], 63] = False
    assert torch.equal(kcd.cpu()[rows], kc[rows]) and torch.equal(vcd.cpu()[rows], vc[rows])
    assert not torch.equal(kcd.cpu(), kc)


def test_cu_seqlens_past_the_rows_is_reported():
    H, Hkv, d = 2, 1, 64
    x, cu, ctx, table, kc, vc = make([4, 4], [0, 0], H, Hkv, d, d, False)
    cu[2] = 12
    ctx[1] = 8
    q, k, v = views(x.to(DEV), H, Hkv, d, d)
    cs = cos_sin_table(64, d).to(DEV)
    qo = vpp.vpp_rope_append(q, k, v, cs, kc.to(DEV), vc.to(DEV), table.to(DEV), cu.to(DEV), ctx.to(DEV))
    assert vpp.vpp_last_device_status() == vpp.VPP_ERR_INVALID
    pos = torch.tensor([0, 1, 2, 3] * 2)
    check_bf16(qo, rotate(views(x, H, Hkv, d, d)[0], pos, cs.cpu(), 0, False), rotate_slack(x, cs), "q_out")


def test_far_positions_use_their_own_row():
    """A row of a million-position table, and a cache slot in its last block."""
    H, Hkv, d, n = 2, 1, 128, 1 << 20
    x, _, _, _, _, _ = make([1], [0], H, Hkv, d, d, False)
    cs = cos_sin_table(n, d)
    table = torch.full((1, n // 64), -1, dtype=torch.int32)
    table[0, -1] = 1
    kc, vc = torch.zeros((2, 64, Hkv, d), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    q, k, v = views(x.to(DEV), H, Hkv, d, d)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    qo = vpp.vpp_rope_append(q, k, v, cs.to(DEV), kc, vc, table.to(DEV), cu, torch.tensor([n], dtype=torch.int32, device=DEV))
    assert vpp.vpp_last_device_status() == 0
    xq, xk, xv = views(x, H, Hkv, d, d)
    pos = torch.tensor([n - 1])
    check_bf16(qo, rotate(xq, pos, cs, 0, False), rotate_slack(x, cs), "q_out")
    check_bf16(kc[1, 63:64], rotate(xk, pos, cs, 0, False), rotate_slack(x, cs), "key")
    assert torch.equal(vc[1, 63].cpu(), xv[0])
    assert not bool(kc[0].any()) and not bool(kc[1, :63].any())


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(fp8):
    """Rows at the far end of more than 2^32 elements of queries, into the last block of as large a cache."""
    H, Hkv, d, n = 64, 8, 128, 70
    T = (1 << 32) // (H * d) + 100
    pool = (1 << 32) // (64 * Hkv * d) + 5
    q = torch.zeros((T, H, d), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device=DEV)
    live = [randn((n, h, d), 60 + h) for h in (H, Hkv, 1)]
    q[T - n:], k[T - n:] = live[0].to(DEV), live[1].to(DEV)
    v = live[2].expand(n, Hkv, d).contiguous()
    vd = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vd[T - n:] = v.to(DEV)
    kc = torch.zeros((pool, 64, Hkv, d), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pool - 1, pool - 3]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([T - n, T], dtype=torch.int32, device=DEV)
    cs = cos_sin_table(n, d)
    scales = (torch.ones(Hkv, device=DEV), torch.ones(Hkv, device=DEV)) if fp8 else ()
    append = vpp.vpp_rope_append_fp8 if fp8 else vpp.vpp_rope_append
    append(q, k, vd, cs.to(DEV), kc, vc, *scales, table, cu, None, q_out=q)
    assert vpp.vpp_last_device_status() == 0
    pos = torch.arange(n)
    check_bf16(q[T - n:], rotate(live[0], pos, cs, 0, False), rotate_slack(live[0], cs), "q")
    got_k = torch.cat([kc[pool - 1], kc[pool - 3, :n - 64]])
    got_v = torch.cat([vc[pool - 1], vc[pool - 3, :n - 64]])
    want = rotate(live[1], pos, cs, 0, False)
    if fp8:
        got_k, got_v = got_k.view(torch.float8_e4m3fn).double().cpu(), got_v.view(torch.float8_e4m3fn).double().cpu()
        # half a step of E4M3, or of its subnormals (2^-9 apart)
        assert bool(((got_k - want).abs() <= HALF_E4M3 * want.abs() + 2.0 ** -10 + 1e-4).all())
        assert bool(((got_v - v.double()).abs() <= HALF_E4M3 * v.double().abs() + 2.0 ** -10).all())
    else:
        check_bf16(got_k, want, rotate_slack(live[1], cs), "key")
        assert torch.equal(got_v.cpu(), v)
