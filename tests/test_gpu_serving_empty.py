"""Calls without rows or sequences through the binding, on the current and on a given stream, eager and captured."""

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def empty_calls(stream):
    H, Hkv, d = 8, 2, 64
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, k = torch.empty((0, H, d), **bf), torch.empty((0, Hkv, d), **bf)
    kc = torch.full((3, 64, Hkv, d), 2.0, **bf)
    k8, one = torch.full((3, 64, Hkv, d), 9, dtype=torch.uint8, device=DEV), torch.ones(Hkv, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    no_table, no_ctx = torch.empty((0, 3), **i32), torch.empty(0, **i32)
    outs = [
        vpp.vpp_prompt_attn(q, k, k, torch.zeros(3, **i32), stream=stream),
        vpp.vpp_prompt_attn(q, k, k, torch.zeros(1, **i32), lse=torch.empty((H, 0), device=DEV), stream=stream),
        vpp.vpp_decode_attn(q, kc, kc, no_table, no_ctx, stream=stream),
        vpp.vpp_decode_attn_fp8(q, k8, k8, one, one, no_table, no_ctx, lse=torch.empty((H, 0), device=DEV), stream=stream),
        vpp.vpp_rope_append(q, k, k, None, kc, kc.clone(), torch.zeros((2, 3), **i32), torch.zeros(3, **i32), stream=stream),
        vpp.vpp_rope_append_fp8(q, k, k, None, k8, k8.clone(), one, one, no_table, torch.zeros(1, **i32), no_ctx, stream=stream),
    ]
    assert all(o.shape == (0, H, d) for o in outs)
    return kc, k8


@pytest.mark.parametrize("given", [False, True])
def test_nothing_to_do(given):
    kc, k8 = empty_calls(torch.cuda.Stream() if given else None)
    torch.cuda.synchronize()
    assert vpp.vpp_last_device_status() == 0
    assert bool((kc == 2).all()) and bool((k8 == 9).all())


def test_all_sequences_empty():
    """Rows of no sequence alone, and decode rows of length 0 alone: nothing is read; padding is left, empty rows are written."""
    H, Hkv, d, T = 8, 2, 64, 200
    q, k = (torch.full((T, h, d), float("nan"), dtype=torch.bfloat16, device=DEV) for h in (H, Hkv))
    out, lse = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((H, T), 7.0, device=DEV)
    cu = torch.zeros(6, dtype=torch.int32, device=DEV)
    vpp.vpp_prompt_attn(q, k, k, cu, out=out, lse=lse)
    kc = torch.full((3, 64, Hkv, d), 2.0, dtype=torch.bfloat16, device=DEV)
    qo = torch.full_like(q, 7.0)
    vpp.vpp_rope_append(q, k, k, None, kc, kc.clone(), torch.full((5, 3), -1, dtype=torch.int32, device=DEV), cu, q_out=qo)
    o = vpp.vpp_decode_attn(q, kc, kc, torch.full((T, 3), -1, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV))
    assert vpp.vpp_last_device_status() == 0
    assert bool((out == 7).all()) and bool((lse == 7).all()) and bool((qo == 7).all()) and bool((kc == 2).all()) and not bool(o.any())


def test_a_given_stream_is_the_current_one_of_a_block():
    """stream= and `with torch.cuda.stream` together, the same and different ones: results as on one stream."""
    H, Hkv, d, n = 8, 2, 64, 300
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn((n, h, d), generator=g, device=DEV, dtype=torch.bfloat16) for h in (H, Hkv, Hkv))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    want = vpp.vpp_prompt_attn(q, k, v, cu)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        for current, given in ((a, a), (a, b), (b, a)):
            with torch.cuda.stream(current):
                o = vpp.vpp_prompt_attn(q, k, v, cu, stream=given)
                current.wait_stream(given)
                got.append(o.clone())
                del o
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
