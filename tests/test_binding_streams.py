"""Memory that the binding allocates for a call on a given stream comes from that stream's pool: a block of the caller's current
stream may still be in use by work queued there, which the given stream does not wait for."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp

DEV = "cuda"


class Block:
    """A tensor's fields as the binding reads them, the stream it was allocated on and those it was recorded on."""

    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype, on=None):
        self.shape, self.dtype, self.on, self.recorded = tuple(shape) if not isinstance(shape, int) else (shape,), dtype, on, []

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 16

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded.append(stream)


class Anything:
    """A library (or call module) whose functions accept everything: sizes are 4096, statuses 0."""

    def __getattr__(self, name):
        return lambda *a: 4096 if "size" in name else 0


@pytest.fixture
def allocations(monkeypatch):
    """The blocks that a call allocates, with streams given by name and "caller" the current one."""
    current, made = ["caller"], []

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(shape, dtype=None, device=None):
        made.append(Block(shape, dtype, current[-1]))
        return made[-1]

    stream = SimpleNamespace(cuda_stream=7)
    monkeypatch.setattr(vpp.torch, "empty", empty)
    monkeypatch.setattr(vpp.torch.cuda, "stream", use)
    monkeypatch.setattr(vpp.torch.cuda, "current_stream", lambda device=None: current[-1] if current[-1] != "caller" else SimpleNamespace(
        cuda_stream=0, name="caller"))
    monkeypatch.setattr(vpp.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(vpp.torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(vpp, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(vpp, "load", Anything)
    monkeypatch.setattr(vpp, "_calls", Anything)
    return stream, made


BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def calls():
    q, k3, c4, c8 = Block((5, 8, 128), BF), Block((5, 4, 128), BF), Block((9, 64, 4, 128), BF), Block((9, 64, 4, 128), U8)
    flat, sc, bt, i1, i2 = Block((64, 4, 128), BF), Block((4,), F32), Block((5, 3), I32), Block((5,), I32), Block((5, 16), I32)
    cu, ctx = [0, 5], [5]
    return {
        "vpp_chunk_attn": (q, flat, flat, 3),
        "vpp_chunk_attn_ex": (q, c4, c4, 3, bt),
        "vpp_chunk_attn_noalloc": (q, c4, c4, 3, bt),
        "vpp_mixed_attn": (q, c4, c4, bt, cu, ctx),
        "vpp_chunk_attn_fp8": (q, c8, c8, sc, sc, 3, bt),
        "vpp_mixed_attn_fp8": (q, c8, c8, sc, sc, bt, cu, ctx),
        "vpp_topk_chunk_attn": (q, c4, c4, 3, i2, i1, bt),
        "vpp_topk_chunk_attn_fp8": (q, c8, c8, sc, sc, 3, i2, i1, bt),
        "vpp_rope_append": (q, k3, k3, None, c4, c4, bt, i1),
        "vpp_rope_append_fp8": (q, k3, k3, None, c8, c8, sc, sc, bt, i1),
        "vpp_decode_attn": (q, c4, c4, bt, i1),
        "vpp_decode_attn_fp8": (q, c8, c8, sc, sc, bt, i1),
        "vpp_prompt_attn": (q, k3, k3, i1),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_a_given_stream_allocates_from_its_own_pool(allocations, monkeypatch, name):
    stream, made = allocations
    monkeypatch.setattr(vpp, "_ptr", lambda t: 0)
    out = getattr(vpp, name)(*calls()[name], stream=stream)
    assert made and out in made
    assert all(b.on is stream for b in made), [b.on for b in made]
    # the caller reads the output on its own stream: freed there, it must not be written again before
    assert [getattr(s, "name", s) for s in out.recorded] == ["caller"]
    # a workspace is used on the given stream alone, whose order is enough for its memory's next use
    assert not any(b.recorded for b in made if b is not out)


@pytest.mark.parametrize("name", list(calls()))
def test_without_a_stream_the_current_pool_serves(allocations, monkeypatch, name):
    _, made = allocations
    monkeypatch.setattr(vpp, "_ptr", lambda t: 0)
    out = getattr(vpp, name)(*calls()[name])
    assert out in made and all(b.on == "caller" and not b.recorded for b in made)


def _operands(H=16, Hkv=4, d=128, n=700):
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn((n, h, d), generator=g, device=DEV, dtype=torch.bfloat16) for h in (H, Hkv, Hkv))
    pages = (n + 63) // 64
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None].expand(n, pages).contiguous()
    kc, vc = torch.zeros((pages, 64, Hkv, d), dtype=torch.bfloat16, device=DEV), torch.zeros((pages, 64, Hkv, d), dtype=torch.bfloat16, device=DEV)
    vpp.vpp_kv_append(k, v, kc, vc, 0, block_table=table[0])
    lens = torch.arange(1, n + 1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    cs, ko = torch.randn((n, d), generator=g, device=DEV), torch.empty_like(k)
    return {
        "prompt": lambda s: vpp.vpp_prompt_attn(q, k, v, cu, stream=s),
        "decode": lambda s: vpp.vpp_decode_attn(q, kc, vc, table, lens, stream=s),
        "rope": lambda s: vpp.vpp_rope_append(q, k, None, cs, None, None, None, cu, k_out=ko, stream=s),
        "chunk": lambda s: vpp.vpp_chunk_attn_ex(q, kc, vc, 0, block_table=table[0], stream=s),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["prompt", "decode", "rope", "chunk"])
def test_queued_work_on_the_current_stream_keeps_its_blocks(name):
    """A block that was freed while work on the current stream still reads it is not what a call on another stream writes."""
    call = _operands()[name]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    big = torch.zeros(1 << 29, device=DEV)  # 2 GB
    src = torch.randint(0, 255, (want.numel() * want.element_size(),), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        blocks = [src.clone() for _ in range(4)]  # of the output's size
        torch.cuda.synchronize()
        for _ in range(60):
            big.add_(1.0)  # keeps the current stream busy for tens of milliseconds
        copies = [b.clone() for b in blocks]
        addresses = {b.data_ptr() for b in blocks}
        del blocks
        got = [call(side) for _ in range(4)]
        assert not addresses & {o.data_ptr() for o in got}
        torch.cuda.synchronize()
        assert all(torch.equal(c, src) for c in copies)
        assert all(torch.equal(o, want) for o in got)
    assert vpp.vpp_last_device_status() == 0
