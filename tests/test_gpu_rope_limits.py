"""Rotate-and-append where a CTA serves several tokens (from about 1200 tokens two, from about 2400 four), at the largest head
dims, and what it stores for the decode call beside it."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_E4M3, rotate, rotate_slack
from tests.test_gpu_rope_append import SHAPES, check_bf16, cos_sin_table, make, slots, views

pytestmark = pytest.mark.gpu
DEV = "cuda"

WIDE = [
    # H, Hkv, dq, dv, rot, start, interleaved
    (3, 1, 320, 64, 64, 128, True),    # 20 tasks a row: threads of a token without a row
    (2, 2, 448, 320, 448, 0, False),   # 28 tasks
    (2, 1, 512, 512, 512, 0, True),
    (4, 2, 512, 64, 16, 8, False),
    (1, 1, 384, 448, 128, 200, False),
]
FEW = ([1, 0, 63, 64, 2, 130, 1, 5], [0, 9, 1, 0, 126, 3, 1000, 61])
SOME = ([700, 1, 0, 640, 64, 95], [0, 500, 7, 63, 1, 129])
MANY = ([3000, 1499, 1, 500], [0, 62, 4000, 1])


def check(new, past, shape, fp8, pad):
    H, Hkv, dq, dv, rot, start, il = shape
    x, cu, ctx, table, kc, vc = make(new, past, H, Hkv, dq, dv, fp8, pad=pad)
    q, k, v = views(x, H, Hkv, dq, dv)
    cs = cos_sin_table(int(ctx.max()), rot) if rot else None
    ks, vs = (0.01 + 0.02 * torch.rand(Hkv, generator=torch.Generator().manual_seed(i)) for i in (1, 2))
    xd = x.to(DEV)
    qd, kd, vd = views(xd, H, Hkv, dq, dv)
    kcd, vcd = kc.to(DEV), vc.to(DEV)
    qo = torch.full((x.shape[0], H, dq), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((x.shape[0], Hkv, dq), 7.0, dtype=torch.bfloat16, device=DEV)
    scales = (ks.to(DEV), vs.to(DEV)) if fp8 else ()
    append = vpp.vpp_rope_append_fp8 if fp8 else vpp.vpp_rope_append
    append(qd, kd, vd, None if cs is None else cs.to(DEV), kcd, vcd, *scales, table.to(DEV), cu.to(DEV), ctx.to(DEV), q_out=qo,
           k_out=ko, rot_start=start, interleaved=il)
    assert vpp.vpp_last_device_status() == 0
    assert torch.equal(xd.cpu(), x), "inputs changed"
    t, pos, blk, row = slots(cu, ctx, table)
    slack = rotate_slack(x, cs)
    rk = rotate(k[t], pos, cs, start, il)
    check_bf16(qo.cpu()[t], rotate(q[t], pos, cs, start, il), slack, "q_out")
    check_bf16(ko.cpu()[t], rk, slack, "k_out")
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
    if fp8:  # values are not rotated: their codes are the rounded quotients, exactly
        want = (v[t].float() / vs[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(vcd.cpu()[blk, row], want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES + WIDE, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("batch", [SOME, MANY], ids=["some", "many"])
def test_several_tokens_a_cta(shape, batch, fp8):
    check(*batch, shape, fp8, 41)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "-".join(map(str, s)))
def test_large_head_dims(shape, fp8):
    check(*FEW, shape, fp8, 3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", [(1024, 1024, 64, 64, 64, 0, False), (16384, 1024, 64, 64, 32, 32, True), (512, 512, 512, 512, 512, 0, False)],
                         ids=lambda s: "-".join(map(str, s)))
def test_many_heads(shape, fp8):
    check([1, 3], [70, 0], shape, fp8, 1)


def test_values_of_an_e4m3_step_are_the_ones_given():
    """Prompts, then decode steps: the codes in the cache are those of the values, token by token, and the attention over the
    cache is that of the values to E4M3's precision."""
    H, Hkv, d = 8, 2, 64
    lens = [61, 5, 130]
    B, T = len(lens), sum(lens)
    cs = cos_sin_table(256, d).to(DEV)
    table = torch.randperm(B * 3, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(B, 3).to(DEV)
    kc = torch.zeros((B * 3, 64, Hkv, d), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks, vs = torch.tensor([0.03, 0.02], device=DEV), torch.tensor([0.02, 0.01], device=DEV)
    x = torch.randn((T, (H + 2 * Hkv) * d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    q, k, v = views(x.to(DEV), H, Hkv, d, d)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    vpp.vpp_rope_append_fp8(q, k, v, cs, kc, vc, ks, vs, table, cu)
    vals = [v.cpu()[int(cu[b]):int(cu[b + 1])] for b in range(B)]
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    one = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    for i in range(4):
        y = torch.randn((B, (H + 2 * Hkv) * d), generator=torch.Generator().manual_seed(6 + i)).to(torch.bfloat16)
        q, k, v = views(y.to(DEV), H, Hkv, d, d)
        ctx += 1
        vpp.vpp_rope_append_fp8(q, k, v, cs, kc, vc, ks, vs, table, one, ctx)
        vals = [torch.cat([a, v.cpu()[b:b + 1]]) for b, a in enumerate(vals)]
    assert vpp.vpp_last_device_status() == 0
    for b in range(B):
        n = int(ctx[b])
        pos = torch.arange(n)
        got = vc.cpu()[table.cpu()[b].long()[pos // 64], pos % 64]
        want = (vals[b].float() / vs.cpu()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(got, want.view(torch.uint8))
        back = got.view(torch.float8_e4m3fn).double() * vs.cpu().double()[:, None]
        assert bool(((back - vals[b].double()).abs() <= HALF_E4M3 * vals[b].double().abs() + 2.0 ** -10 * vs.cpu().double()[:, None] * 1.01).all())
