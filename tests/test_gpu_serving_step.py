"""The serving operators run together, as a model's step would call them: a
batch of prompts, then captured decode steps whose lengths grow on the device."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, HALF_F16, attend, check_attention, randn, rotate
from tests.test_gpu_rope_append import cos_sin_table, views

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_then_captured_decode_steps(fp8):
    H, Hkv, d, steps = 8, 2, 128, 6
    lens = [61, 5, 130, 64]
    B, T = len(lens), sum(lens)
    cs = cos_sin_table(512, d)
    csd = cs.to(DEV)
    maxb = 4
    table = torch.randperm(B * maxb, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(B, maxb).to(DEV)
    kc = torch.zeros((B * maxb, 64, Hkv, d), dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    scales = (torch.full((Hkv,), 0.03, device=DEV), torch.full((Hkv,), 0.02, device=DEV)) if fp8 else ()
    append = vpp.vpp_rope_append_fp8 if fp8 else vpp.vpp_rope_append
    decode = vpp.vpp_decode_attn_fp8 if fp8 else vpp.vpp_decode_attn

    # the prompts: rotate in place and fill the cache, then attend over the packed projection
    x = randn((T, (H + 2 * Hkv) * d), 1).to(DEV)
    q, k, v = views(x, H, Hkv, d, d)
    q0, k0, v0 = (t.clone().cpu() for t in (q, k, v))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    append(q, k, v, csd, kc, vc, *scales, table, cu, None, q_out=q, k_out=k)
    out = vpp.vpp_prompt_attn(q, k, v, cu)
    assert vpp.vpp_last_device_status() == 0
    at = 0
    keys, vals = [], []
    for n in lens:
        rows = slice(at, at + n)
        pos = torch.arange(n)
        assert float((q[rows].cpu().double() - rotate(q0[rows], pos, cs, 0, False)).abs().max()) < 0.05
        ref = attend(q[rows].cpu(), k[rows].cpu(), v0[rows], d ** -0.5, True)
        check_attention(out[rows], None, ref, d, HALF_BF16, "prompt")
        keys.append(rotate(k0[rows], pos, cs, 0, False))
        vals.append(v0[rows].double())
        at += n

    # decode steps: one captured graph, lengths advanced on the device
    y = torch.zeros((B, (H + 2 * Hkv) * d), dtype=torch.bfloat16, device=DEV)
    qs, kn, vn = views(y, H, Hkv, d, d)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    one = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    qr = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV)
    o, lse = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((H, B), device=DEV)
    ws = torch.empty(vpp.decode_attn_workspace_size(B, H, Hkv, d, d) + 16, dtype=torch.uint8, device=DEV)

    def step():
        ctx.add_((ctx > 0).to(torch.int32))
        append(qs, kn, vn, csd, kc, vc, *scales, table, one, ctx, q_out=qr)
        decode(qr, kc, vc, *scales, table, ctx, out=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = [t.clone() for t in (kc, vc, ctx)]
    with torch.cuda.stream(side):
        step()  # warm-up, undone below
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip((kc, vc, ctx), before):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    now = list(lens)
    for i in range(steps):
        if i == 3:  # a sequence ends: its row becomes padding
            ctx[1] = 0
            now[1] = 0
        fresh = randn((B, (H + 2 * Hkv) * d), 50 + i)
        y.copy_(fresh)
        graph.replay()
        now = [n + 1 if n else 0 for n in now]
        fq, fk, fv = views(fresh, H, Hkv, d, d)
        for b in range(B):
            if now[b] == 0:
                assert not bool(o[b].any()) and bool((lse[:, b] == -float("inf")).all())
                continue
            pos = torch.tensor([now[b] - 1])
            keys[b] = torch.cat([keys[b], rotate(fk[b:b + 1], pos, cs, 0, False)])
            vals[b] = torch.cat([vals[b], fv[b:b + 1].double()])
            got_k, got_v = (torch.stack([c[int(table[b, p // 64]), p % 64] for p in range(now[b])]).cpu() for c in (kc, vc))
            if fp8:
                got_k = got_k.view(torch.float8_e4m3fn).double() * 0.03 * (1.0)
                got_v = got_v.view(torch.float8_e4m3fn).double() * 0.02
                got_k, got_v = got_k * (float(scales[0][0]) / 0.03), got_v * (float(scales[1][0]) / 0.02)
                # E4M3 holds a value to half a step
                assert bool(((got_k - keys[b]).abs() <= 2.0 ** -4 * keys[b].abs() + 0.03 * 2.0 ** -10 + 1e-5).all())
            else:
                assert bool(((got_k.double() - keys[b]).abs() <= HALF_BF16 * keys[b].abs() + 1e-5).all())
                assert torch.equal(got_v.double(), vals[b])
            ref = attend(qr[b:b + 1].cpu(), got_k, got_v, d ** -0.5, False)
            check_attention(o[b:b + 1], lse[:, b:b + 1], ref, d, HALF_F16 if fp8 else HALF_BF16, f"step {i}, row {b}")
    assert vpp.vpp_last_device_status() == 0


def test_prompts_and_decode_agree():
    """The last token of each prompt, as a decode row over the cache the prompts were appended to, gives what prompt
    attention gives it."""
    H, Hkv, d = 12, 4, 64
    lens = [1, 64, 200, 77]
    T, B = sum(lens), len(lens)
    x = randn((T, (H + 2 * Hkv) * d), 3).to(DEV)
    q, k, v = views(x, H, Hkv, d, d)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    table = torch.arange(B * 4, dtype=torch.int32, device=DEV).view(B, 4)
    kc = torch.zeros((B * 4, 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    vpp.vpp_rope_append(q, k, v, cos_sin_table(256, d).to(DEV), kc, vc, table, cu, q_out=q, k_out=k)
    lse = torch.empty((H, T), device=DEV)
    out = vpp.vpp_prompt_attn(q, k, v, cu, lse=lse)
    last = (cu[1:] - 1).long()
    lse1 = torch.empty((H, B), device=DEV)
    one = vpp.vpp_decode_attn(q[last], kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV), lse=lse1)
    at = 0
    for b, n in enumerate(lens):
        ref = attend(q[at + n - 1:at + n].cpu(), k[at:at + n].cpu(), v[at:at + n].cpu(), d ** -0.5, False)
        check_attention(one[b:b + 1], lse1[:, b:b + 1], ref, d, HALF_BF16, "decode")
        check_attention(out[at + n - 1:at + n], lse[:, at + n - 1:at + n], ref, d, HALF_BF16, "prompt")
        at += n


def test_a_captured_step_on_forked_streams():
    """The calls of a step captured on two streams that fork and join, between copies and fills: every call sees what the
    ones before it wrote, in each of many replays."""
    H, Hkv, d, B = 16, 4, 128, 6
    lens = [40, 200, 1, 129, 64, 300]
    T = sum(lens)
    cs = cos_sin_table(512, d).to(DEV)
    x0 = [randn((T, (H + 2 * Hkv) * d), 70 + i).to(DEV) for i in range(3)]
    x = torch.zeros_like(x0[0])
    q, k, v = views(x, H, Hkv, d, d)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    last = (cu[1:] - 1).long()
    table = torch.randperm(B * 5, generator=torch.Generator().manual_seed(9)).to(torch.int32).view(B, 5).to(DEV)
    kc = torch.zeros((B * 5, 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    qr, kr = torch.empty((T, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((T, Hkv, d), dtype=torch.bfloat16, device=DEV)
    out, o = torch.empty((T, H, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(vpp.decode_attn_workspace_size(B, H, Hkv, d, d) + 16, dtype=torch.uint8, device=DEV)
    ql = torch.empty((B, H, d), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        kc.zero_()
        vc.fill_(0)
        vpp.vpp_rope_append(q, k, v, cs, kc, vc, table, cu, q_out=qr, k_out=kr)
        side.wait_stream(main)
        vpp.vpp_prompt_attn(qr, kr, v, cu, out=out)
        with torch.cuda.stream(side):
            ql.copy_(qr[last])
            vpp.vpp_decode_attn(ql, kc, vc, table, ctx, out=o, workspace=ws)
            vpp.vpp_decode_attn(ql, kc, vc, table, ctx, out=o, workspace=ws)
        main.wait_stream(side)
        vpp.vpp_prompt_attn(qr, kr, v, cu, out=out)
        qr.zero_()

    def run(i):
        x.copy_(x0[i])

    want = []
    for i in range(3):
        run(i)
        step()
        torch.cuda.synchronize()
        want.append((out.clone(), o.clone()))
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 2, 1, 0, 2):
        run(i)
        out.zero_(), o.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(o, want[i][1])
    assert vpp.vpp_last_device_status() == 0
    # and the step itself is right, on the rotated rows as the append wrote them
    run(2)
    vpp.vpp_rope_append(q, k, v, cs, kc, vc, table, cu, q_out=qr, k_out=kr)
    for b, n in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b]) + n)
        ref = attend(qr[rows].cpu(), kr[rows].cpu(), v[rows].cpu(), d ** -0.5, True)
        check_attention(want[2][0][rows], None, ref, d, HALF_BF16, f"prompt {b}")
        tail = tuple(t[-1:] if i % 2 == 0 else t[:, -1:] for i, t in enumerate(ref))
        check_attention(want[2][1][b:b + 1], None, tail, d, HALF_BF16, f"decode row {b}")
