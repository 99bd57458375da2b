"""Decode over an E4M3 cache where most of a row's weight vector is far below its largest entry: one dominant key whose value is
zero, so that the result is the tail's alone."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import HALF_BF16, HALF_F16, attend

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("at", [0, 517])  # where the dominant key is: at the start, or after the maximum has been set by others
@pytest.mark.parametrize("depth", [6, 10, 12, 14, 16, 18, 20])  # nats between it and the others; E4M3 values
@pytest.mark.parametrize("H,Hkv,n", [(456, 456, 1024), (32, 2, 4096)])
def test_a_tail_below_a_dominant_key_keeps_its_weight(H, Hkv, n, depth, at):
    d = 64
    g = torch.Generator().manual_seed(depth)
    k = torch.zeros((n, Hkv, d))
    k[:, :, 0] = -float(depth)
    k[at] = 0.0
    v = (0.5 + 0.5 * torch.rand((n, Hkv, d), generator=g)).to(torch.float8_e4m3fn)
    v[at] = 0.0
    k = k.to(torch.float8_e4m3fn)
    q = torch.zeros((1, H, d), dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    pages = n // 64
    kc, vc = (x.view(torch.uint8).reshape(pages, 64, Hkv, d).to(DEV) for x in (k, v))
    one = torch.ones(Hkv, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    lse = torch.empty((H, 1), device=DEV)
    out = vpp.vpp_decode_attn_fp8(q.to(DEV), kc, vc, one, one, table, ctx, lse=lse, softmax_scale=1.0)
    assert vpp.vpp_last_device_status() == 0
    o, l, absw, mag = attend(q, k.double(), v.double(), 1.0, False)
    # The scores are exact (one product of small whole numbers), so a weight is off by its float32 exponential only: 2^-22 for
    # the instruction, 2^-24 |s log2 e| for each of its argument's two roundings.  P's rounding to f16 is 2^-11 of the weight or,
    # below f16's normal range, half of 2^-24: the largest weight is 2^14 at least in f16, so 2^-39 of it.  Sums as in
    # check_attention; one rounding to bf16.
    ds = 2.0 ** -22 + 2 * 2.0 ** -24 * depth * 1.4427
    top = (torch.zeros_like(l) - l).exp().t()[..., None]  # the dominant key's weight
    sum_v = v.double().abs().sum(0).repeat_interleave(H // Hkv, 0)[None]
    tol = HALF_BF16 * o.abs() + ((HALF_F16 + 2 * ds + 2.0 ** -16) * absw + 2.0 ** -39 * top * sum_v) * (1 + HALF_BF16)
    worst = float(((out.double().cpu() - o).abs() / tol).max())
    assert worst <= 1.0, f"off by {worst:.3f} of the tolerance"
    assert float((lse.double().cpu() - l).abs().max()) <= 2.0 ** -16 + 2.0 ** -22 * float(l.abs().max())


@pytest.mark.parametrize("power", [120, 100, 76, 75, 60, 0, -40, -60, -90, -110])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (12, 1, 64)])
def test_queries_of_any_size(H, Hkv, d, power):
    """Queries scaled by a power of two and a softmax scale that takes it back give the rows of the unscaled ones: they are
    exact multiples in bf16, and the scores differ by nothing."""
    g = torch.Generator().manual_seed(1)
    n = 300
    kc, vc = (torch.randn((5, 64, Hkv, d), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for _ in range(2))
    q = torch.randn((2, H, d), generator=g).to(torch.bfloat16).double()
    one = torch.ones(Hkv, device=DEV)
    table = torch.arange(5, dtype=torch.int32, device=DEV).expand(2, 5).contiguous()
    ctx = torch.tensor([n, 17], dtype=torch.int32, device=DEV)
    got = []
    for e in (0, power):
        lse = torch.empty((H, 2), device=DEV)
        out = vpp.vpp_decode_attn_fp8((q * 2.0 ** e).to(torch.bfloat16).to(DEV), kc, vc, one, one, table, ctx, lse=lse, softmax_scale=0.125 * 2.0 ** -e)
        got.append((out.cpu(), lse.cpu()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
