"""Refusals of the device-planned serving operators: arguments are checked on
the host before any launch, so these run without a GPU."""

import ctypes

import pytest

from chunked_prefill_causal_gb300 import vpp

P = 0x100000  # a 16-byte aligned address, never dereferenced: validation fails first
BAD = P + 8


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return vpp.load()


ROPE = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, cs=P, rows=64, start=0, rot=64, il=0, qo=P + 4096, qos=512, ko=None, kos=0,
            kc=P, vc=P, bt=P, mb=4, nb=8, cu=P, ctx=P, batch=2, T=5, H=8, Hkv=4, dq=64, dv=64, st=None)
DEC = dict(q=P, qs=512, kc=P, vc=P, bt=P, mb=4, nb=8, ctx=P, batch=2, H=8, Hkv=4, dq=64, dv=64, scale=0.0, out=P, lse=P, ws=P, wb=1 << 40,
           st=None)
PRO = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, cu=P, batch=2, T=5, H=8, Hkv=4, dq=64, dv=64, scale=0.0, out=P, lse=P, st=None)


def args(base, change):
    assert set(change) <= set(base)
    return [{**base, **change}[n] for n in base]


INV, UNS = vpp.VPP_ERR_INVALID, vpp.VPP_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,code", [
    (dict(k=None), INV), (dict(k=BAD), INV), (dict(q=BAD), INV), (dict(v=BAD), INV), (dict(qo=None), INV), (dict(qo=BAD), INV),
    (dict(q=None), INV),  # q_out without q
    (dict(qs=504), INV), (dict(qs=516), INV), (dict(ks=248), INV), (dict(vs=252), INV), (dict(qos=256), INV), (dict(ks=-256), INV),
    (dict(qo=P, qos=1024), INV),  # in place needs the same stride
    (dict(ko=P, kos=512), INV), (dict(ko=BAD, kos=256), INV), (dict(ko=P + 64, kos=128), INV),
    (dict(cs=None), INV), (dict(cs=BAD), INV), (dict(rows=0), INV), (dict(rot=-16), INV), (dict(start=8), INV), (dict(rot=80), INV),
    (dict(rot=24), UNS), (dict(rot=32, start=4), UNS), (dict(start=-8, rot=16), INV),
    (dict(cu=None), INV), (dict(cu=P + 2), INV), (dict(ctx=P + 1), INV), (dict(batch=0), INV), (dict(batch=-1), INV), (dict(T=-1), INV),
    (dict(T=1 << 31), INV), (dict(H=0), INV), (dict(Hkv=0), INV), (dict(dq=96), UNS), (dict(dv=96), UNS), (dict(dq=576), UNS),
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(kc=BAD), INV), (dict(bt=None), INV), (dict(bt=P + 2), INV), (dict(mb=0), INV),
    (dict(nb=0), INV), (dict(kc=None, vc=None), INV),  # rotation only, without k_out
])
def test_rope_append_refuses(lib, change, code):
    assert lib.vpp_rope_append(*args(ROPE, change)) == code
    names = list(ROPE)
    fp8 = args(ROPE, change)
    at = names.index("bt")
    assert lib.vpp_rope_append_fp8(*fp8[:at], P, P, *fp8[at:]) == code


def test_rope_append_fp8_needs_scales_and_a_cache(lib):
    names, a = list(ROPE), args(ROPE, {})
    at = names.index("bt")
    assert lib.vpp_rope_append_fp8(*a[:at], None, P, *a[at:]) == INV
    assert lib.vpp_rope_append_fp8(*a[:at], P, P + 2, *a[at:]) == INV
    b = args(ROPE, dict(kc=None, vc=None, ko=P + 64, kos=256))
    assert lib.vpp_rope_append_fp8(*b[:at], P, P, *b[at:]) == INV


@pytest.mark.parametrize("change,code", [
    (dict(q=None), INV), (dict(q=BAD), INV), (dict(qs=504), INV), (dict(qs=516), INV), (dict(kc=None), INV), (dict(vc=BAD), INV),
    (dict(bt=None), INV), (dict(mb=0), INV), (dict(nb=0), INV), (dict(mb=1 << 26), INV), (dict(ctx=None), INV), (dict(ctx=P + 2), INV),
    (dict(batch=-1), INV), (dict(H=7), INV), (dict(H=0), INV), (dict(Hkv=0), INV), (dict(H=68, Hkv=4, qs=68 * 64), UNS), (dict(dq=96), UNS),
    (dict(dq=256), UNS), (dict(dv=192), UNS), (dict(out=None), INV), (dict(out=BAD), INV), (dict(lse=P + 2), INV),
])
def test_decode_refuses(lib, change, code):
    a = args(DEC, change)
    assert lib.vpp_decode_attn(*a) == code
    assert lib.vpp_decode_attn_fp8(*a[:4], P, P, *a[4:]) == code


def test_decode_fp8_needs_scales(lib):
    a = args(DEC, {})
    assert lib.vpp_decode_attn_fp8(*a[:4], None, P, *a[4:]) == INV
    assert lib.vpp_decode_attn_fp8(*a[:4], P, None, *a[4:]) == INV


@pytest.mark.parametrize("change,code", [
    (dict(q=None), INV), (dict(k=BAD), INV), (dict(v=None), INV), (dict(qs=504), INV), (dict(ks=260), INV), (dict(vs=128), INV),
    (dict(cu=None), INV), (dict(cu=P + 2), INV), (dict(batch=0), INV), (dict(batch=-2), INV), (dict(T=-5), INV), (dict(T=1 << 31), INV),
    (dict(H=9), INV), (dict(H=68, Hkv=4, qs=68 * 64), UNS), (dict(dq=32), UNS), (dict(dv=192), UNS), (dict(out=None), INV), (dict(out=BAD), INV),
    (dict(lse=P + 1), INV),
])
def test_prompt_refuses(lib, change, code):
    assert lib.vpp_prompt_attn(*args(PRO, change)) == code


def test_empty_calls_are_no_ops(lib):
    assert lib.vpp_rope_append(*[None if n in ("q", "k", "v", "cs", "qo", "kc", "vc", "bt", "cu", "ctx") else v
                                 for n, v in {**ROPE, "T": 0}.items()]) == vpp.VPP_OK
    assert lib.vpp_decode_attn(*args(DEC, dict(batch=0, q=None, kc=None, vc=None, bt=None, ctx=None, out=None, lse=None))) == vpp.VPP_OK
    assert lib.vpp_prompt_attn(*args(PRO, dict(T=0, q=None, k=None, v=None, cu=None, out=None, lse=None))) == vpp.VPP_OK


def test_workspace_sizes(lib):
    assert vpp.decode_attn_workspace_size(0, 8, 2, 128, 128) == 0
    assert vpp.decode_attn_workspace_size(4, 7, 2, 128, 128) == 0
    assert vpp.decode_attn_workspace_size(4, 8, 2, 96, 128) == 0
    assert vpp.decode_attn_workspace_size(1, 8, 2, 128, 128) >= 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("covers the check without a GPU")
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
        vpp.vpp_prompt_attn(x, x, x, torch.zeros(2, dtype=torch.int32))
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def fake(*shape, dtype=None, stride=None):
    """A host tensor of this shape and stride; the call module takes them for device -1."""
    import torch
    dtype = dtype or torch.bfloat16
    return torch.zeros(shape, dtype=dtype) if stride is None else torch.empty_strided(shape, stride, dtype=dtype)


def test_the_call_module_checks_tensors(lib):
    """Types, devices, shapes and strides, on host tensors; what passes reaches the library, whose own refusal (head dims
    of 96) comes back as its status before anything is read."""
    torch = pytest.importorskip("torch")
    c = vpp._calls()
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8

    def prompt(dev=-1, **kw):
        a = dict(q=fake(5, 8, 96), k=fake(5, 4, 96), v=fake(5, 4, 64), cu=fake(3, dtype=i32), out=fake(5, 8, 64), lse=fake(8, 5, dtype=f32))
        return c.prompt(dev, 0, *{**a, **kw}.values(), 0.0)

    assert prompt() == UNS and prompt(lse=None) == UNS
    assert prompt(q=fake(5, 8, 96, stride=(2000, 96, 1))) == UNS  # part of a wider projection
    bad = [dict(q=fake(5, 8, 96, dtype=f32)), dict(dev=0), dict(dev=1), dict(q=fake(5, 768)),
           dict(q=fake(5, 8, 96, stride=(768, 1, 8))), dict(q=fake(5, 8, 96, stride=(800, 100, 1))), dict(k=fake(4, 4, 96)), dict(k=fake(5, 4, 64)),
           dict(k=fake(5, 2, 96)), dict(v=fake(6, 4, 64)), dict(cu=fake(3, dtype=torch.int64)), dict(cu=fake(3, dtype=i32, stride=(2,))),
           dict(cu=fake(3, 1, dtype=i32)), dict(out=fake(5, 8, 96)), dict(out=fake(5, 8, 64, stride=(1024, 64, 1))), dict(lse=fake(5, 8, dtype=f32)),
           dict(lse=fake(8, 5))]
    for b in bad:
        with pytest.raises(ValueError):
            prompt(**b)

    def decode(dev=-1, **kw):
        a = dict(q=fake(3, 8, 96), kc=fake(6, 64, 4, 96), vc=fake(6, 64, 4, 64), ks=None, vs=None, table=fake(3, 4, dtype=i32),
                 ctx=fake(3, dtype=i32), out=fake(3, 8, 64), lse=fake(8, 3, dtype=f32))
        return c.decode(dev, 0, *{**a, **kw}.values(), 0.0, 0, 0)

    fp8 = dict(kc=fake(6, 64, 4, 96, dtype=u8), vc=fake(6, 64, 4, 64, dtype=u8), ks=fake(4, dtype=f32), vs=fake(4, dtype=f32))
    assert decode() == UNS and decode(**fp8) == UNS
    bad = [dict(q=fake(3, 8, 64)), dict(kc=fake(6, 32, 4, 96)), dict(vc=fake(5, 64, 4, 64)), dict(vc=fake(6, 64, 2, 64)), dict(kc=fp8["kc"]),
           dict(table=fake(2, 4, dtype=i32)), dict(table=fake(3, 4)), dict(table=fake(12, dtype=i32)), dict(ctx=fake(2, dtype=i32)), dict(out=fake(3, 8, 96)),
           dict(lse=fake(3, 8, dtype=f32)), {**fp8, "ks": fake(3, dtype=f32)}, {**fp8, "vs": fake(4)}, {**fp8, "kc": fake(6, 64, 4, 96)}, dict(dev=0)]
    for b in bad:
        with pytest.raises(ValueError):
            decode(**b)
    assert decode(q=fake(3, 8, 96, stride=(1000, 96, 1))) == UNS
    with pytest.raises(ValueError):
        decode(table=torch.empty((3, 1 << 33), dtype=i32, device="meta"))

    def rope(dev=-1, **kw):
        a = dict(q=fake(5, 8, 96), k=fake(5, 4, 96), v=fake(5, 4, 64), cs=fake(32, 64, dtype=f32), kc=fake(6, 64, 4, 96), vc=fake(6, 64, 4, 64), ks=None,
                 vs=None, table=fake(2, 4, dtype=i32), cu=fake(3, dtype=i32), ctx=fake(2, dtype=i32), qo=fake(5, 8, 96), ko=None, start=0, il=False)
        return c.rope(dev, 0, *{**a, **kw}.values())

    assert rope() == UNS and rope(ctx=None) == UNS and rope(**fp8) == UNS and rope(q=None, qo=None) == UNS
    assert rope(kc=None, vc=None, v=None, table=None, ko=fake(5, 4, 96)) == UNS
    bad = [dict(q=fake(4, 8, 96)), dict(qo=fake(5, 4, 96)), dict(q=None), dict(k=fake(5, 2, 96)), dict(v=fake(5, 4, 96)), dict(cs=fake(32, 64)), dict(cs=fake(64, dtype=f32)),
           dict(table=fake(3, 4, dtype=i32)), dict(ctx=fake(3, dtype=i32)), dict(ko=fake(5, 8, 96)), dict(kc=fake(6, 64, 4, 64)),
           {**fp8, "ks": fake(3, dtype=f32)}, dict(dev=0)]
    for b in bad:
        with pytest.raises(ValueError):
            rope(**b)
    for f, n in ((c.rope, 17), (c.decode, 14), (c.prompt, 9)):
        with pytest.raises(TypeError):
            f(*[0] * (n - 1))
    with pytest.raises(TypeError):
        c.prompt(0, 0, 1, 2, 3, 4, 5, 6, 0.0)
    with pytest.raises(TypeError):
        prompt(lse=3)
    # a tensor without memory of its own raises a C++ error, which comes back as a Python one
    with pytest.raises((RuntimeError, ValueError)):
        prompt(cu=torch.sparse_coo_tensor(torch.tensor([[0]]), torch.tensor([1], dtype=i32), (3,), check_invariants=True))
