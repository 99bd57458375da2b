"""Captured serving-step calls in the orders that a program may choose: the first call of a process, several graphs, calls on a
given stream inside a capture, other threads' eager calls meanwhile."""

import os
import subprocess
import sys
import threading

import pytest
import torch

from chunked_prefill_causal_gb300 import vpp
from tests.serving_ref import randn
from tests.test_gpu_decode_paged import call, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
from chunked_prefill_causal_gb300 import vpp
H, Hkv, d, T = 8, 2, 64, 130
g = torch.Generator().manual_seed(1)
q, k, v = (torch.randn((T, h, d), generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
cs = torch.randn((256, d), generator=g).cuda()
cu = torch.tensor([0, 100, 130], dtype=torch.int32).cuda()
ctx = torch.tensor([100, 30], dtype=torch.int32).cuda()
table = torch.arange(4, dtype=torch.int32).view(2, 2).cuda()
kc, vc = torch.zeros((4, 64, Hkv, d), dtype=torch.bfloat16).cuda(), torch.zeros((4, 64, Hkv, d), dtype=torch.bfloat16).cuda()
ko = torch.empty_like(k)
torch.cuda.synchronize()

def step():
    qr = vpp.vpp_rope_append(q, k, v, cs, kc, vc, table, cu, k_out=ko)
    return qr, vpp.vpp_prompt_attn(qr, ko, v, cu), vpp.vpp_decode_attn(qr[:2], kc, vc, table, ctx)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
for _ in range(3):
    graph.replay()
torch.cuda.synchronize()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)), "replayed and eager results differ"
assert vpp.vpp_last_device_status() == 0
print("same")
"""


def test_the_first_call_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr


def problem():
    H, Hkv, d = 16, 4, 128
    ctx = [4000, 50, 1700]
    kc, vc, ks, vs, table, _, _ = make(ctx, Hkv, d, d, False)
    return kc, vc, ks, vs, table, torch.tensor(ctx, dtype=torch.int32, device=DEV), [randn((3, H, d), 80 + i).to(DEV) for i in range(3)]


def test_two_graphs_and_eager_calls_replayed_at_once():
    """Two captured calls that were given no workspace, replayed on two streams beside eager calls on a third."""
    kc, vc, ks, vs, table, lens, qs = problem()
    want = [call(False, q, kc, vc, ks, vs, table, lens) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, q in zip(graphs, qs):
        with torch.cuda.graph(g):
            outs.append(call(False, q, kc, vc, ks, vs, table, lens))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager.append(call(False, qs[2], kc, vc, ks, vs, table, lens))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and all(torch.equal(o, want[2]) for o in eager)


def test_a_given_stream_inside_a_capture():
    """A captured fork: calls on a stream given by argument allocate from the graph's memory and keep it between replays."""
    kc, vc, ks, vs, table, lens, qs = problem()
    want = [call(False, q, kc, vc, ks, vs, table, lens) for q in qs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        outs = [call(False, qs[i], kc, vc, ks, vs, table, lens, stream=side) for i in (0, 1)]
        outs.append(call(False, qs[2], kc, vc, ks, vs, table, lens))
        main.wait_stream(side)
    for _ in range(5):
        for o in outs:
            o.zero_()
        junk = [torch.full_like(o, 3.0) for o in outs for _ in range(4)]  # memory that a lost block would come back as
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert all(bool((j == 3.0).all()) for j in junk)


def test_threads_on_their_own_streams():
    """Each thread calls on its own current stream; the workspaces are the threads' own."""
    kc, vc, ks, vs, table, lens, qs = problem()
    want = [call(False, q, kc, vc, ks, vs, table, lens) for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [call(False, qs[i], kc, vc, ks, vs, table, lens) for _ in range(40)]
            torch.cuda.current_stream().synchronize()
            bad.extend(i for o in got if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
