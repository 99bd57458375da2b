"""Refusals of the device-planned serving operators: arguments are checked on
the host before any launch, so these run without a GPU."""

import ctypes
import struct

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


def words(values):
    return b"".join(struct.pack("=f4x", v) if isinstance(v, float) else struct.pack("=q", v or 0) for v in values)


CALLS = [(1, ROPE, {}, "vpp_rope_append"), (3, DEC, {}, "vpp_decode_attn"), (5, PRO, {}, "vpp_prompt_attn")]


@pytest.mark.parametrize("op,base,_,name", CALLS)
def test_packed_call_checks_like_the_call(lib, op, base, _, name):
    """Every argument, spoilt in turn, gives the same answer both ways (without a device, the answer of the good call is
    the missing device's)."""
    for key in [None] + list(base):
        if key == "st":
            continue
        for spoilt in (None, 3, -1, BAD):
            if key is not None and isinstance(base[key], float):
                continue
            a = args(base, {} if key is None else {key: spoilt})
            narrow = key not in (None, "q", "k", "v", "qo", "ko", "kc", "vc", "bt", "cu", "ctx", "out", "lse", "ws", "cs")
            if spoilt is None and narrow or (spoilt == -1 and not narrow) or (key == "wb"):
                continue
            if key is None:
                a = args(base, dict(Hkv=3))  # refused, so that nothing is launched where there is a device
            elif spoilt == 3 and key in ("rows", "mb", "nb", "batch", "T", "il"):
                continue  # a good value: would launch
            elif key in ("ko", "ctx") and spoilt is None or (key == "lse" and spoilt is None):
                continue  # may be missing: would launch
            elif spoilt == BAD and (key == "lse" or key == "ctx" or key == "cu" or key == "bt" or key == "cs" or narrow):
                continue
            want = getattr(lib, name)(*a)
            assert want != vpp.VPP_OK
            assert lib.vpp_call(op, words(a), len(a)) == want, (key, spoilt)


def test_packed_call_refuses_other_counts_and_wide_words(lib):
    for op, base, _, _name in CALLS:
        a = args(base, {})
        assert lib.vpp_call(op, words(a) + bytes(8), len(a) + 1) == INV
        assert lib.vpp_call(op, words(a), len(a) - 1) == INV
        assert lib.vpp_call(op, words(args(base, dict(H=8 + (1 << 32)))), len(a)) == INV
    assert lib.vpp_call(0, words([0] * 40), 29) == INV
    assert lib.vpp_call(9, words([0] * 40), 29) == INV
    assert lib.vpp_call(1, None, 29) == INV


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
