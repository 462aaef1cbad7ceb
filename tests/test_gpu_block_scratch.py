"""Scratch of the operators around the FFN on the GPU: calls on two streams and
from two threads at the same time, and graphs beside calls that need more. All
bit for bit, as each call sums in a fixed order."""

from __future__ import annotations

import importlib.util
import os
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402

DEV = torch.device("cuda", 0)
BF16 = torch.bfloat16

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("transformer_block_scratch",
                                              os.path.join(ROOT, "examples", "transformer_block.py"))
ex = importlib.util.module_from_spec(spec)
sys.modules[spec.name] = ex  # dataclasses look their module up
spec.loader.exec_module(ex)


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(BF16).to(DEV)


def _weights(seed, d, F):
    g = torch.Generator().manual_seed(seed)
    return [_bf16(g, F, d, scale=d**-0.5) for _ in range(3)]


def _jobs(M):
    """One call of each operator that takes scratch, as name -> call."""
    g = torch.Generator().manual_seed(M)
    d, F = 512, 2048
    Wg, Wu, Wd = _weights(3, d, F)
    qg, qu, qd = tw.q4_quantize(Wg), tw.q4_quantize(Wu), tw.q4_quantize(Wd.t().contiguous())
    long = tw.q4_quantize(_bf16(g, 32, 1 << 14, scale=2.0**-7))
    x, xl = _bf16(g, M, d), _bf16(g, M, 1 << 14)
    w, rstd = _bf16(g, d), torch.rand(M, generator=g).to(DEV) + 0.5
    dn = _bf16(g, M, d)
    return {"ffn": lambda: (tw.ffn_forward_q4(x, qg, qu, qd),), "product": lambda: (tw.q4_matmul(xl, long),),
            "pair": lambda: (tw.q4_gateup(xl, long, long),),
            "norm backward": lambda: tw.add_rmsnorm_backward(dn, x, w, rstd)}


def test_two_streams_at_once():
    for name in _jobs(4):
        print(f"[scratch] two streams: {name}", flush=True)
        calls = [_jobs(M)[name] for M in (48, 200)]
        want = [c() for c in calls]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [[], []]
        for _ in range(8):
            for s, c, out in zip(streams, calls, got):
                with torch.cuda.stream(s):
                    out.append(c())
        torch.cuda.synchronize()
        for outs, w in zip(got, want):
            for out in outs:
                assert all(torch.equal(a, b) for a, b in zip(out, w)), name


def test_two_threads_on_one_stream():
    calls = [_jobs(M)["ffn"] for M in (48, 200)]
    want = [c()[0] for c in calls]
    got = [[], []]

    def work(i):
        for _ in range(20):
            got[i].append(calls[i]()[0])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert len(outs) == 20 and all(torch.equal(o, w) for o in outs)


def test_graph_beside_larger_calls():
    """What a graph writes between its calls is its own memory: larger calls,
    fresh allocations and emptied caches neither change its results nor are
    changed by it."""
    d, F, M = 512, 2048, 4
    g = torch.Generator().manual_seed(9)
    layers = [ex.ServedLayer.quantized((1 + 0.1 * torch.randn(d, generator=g)).to(BF16).to(DEV), *_weights(20 + i, d, F))
              for i in range(2)]
    graph, y, h, out = ex.captured(layers, M, d)
    for k in range(4):
        print(f"[scratch] graph, replay {k}", flush=True)
        y0 = torch.randn(M, d, generator=g).to(DEV)
        h0 = _bf16(g, M, d)
        for job in _jobs(64 << k).values():  # each time more than before
            job()
        torch.cuda.empty_cache()
        fresh = [torch.full((1 << n,), 42, dtype=torch.uint8, device=DEV) for n in range(9, 26)]
        y.copy_(y0)
        h.copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        h1 = h0.clone()
        assert torch.equal(out, ex.serve(layers, y0, h1)) and torch.equal(h, h1), k
        assert all((f == 42).all() for f in fresh), k


def test_graph_with_a_workspace_of_the_callers():
    d, M = 512, 48
    call = _jobs(M)
    Wg, Wu, Wd = _weights(3, d, 2048)
    q = tw.q4_quantize(Wg), tw.q4_quantize(Wu), tw.q4_quantize(Wd.t().contiguous())
    x = _bf16(torch.Generator().manual_seed(M), M, d)
    ws = tw.Workspace(DEV)
    ws.get(tw.ffn_q4_workspace_bytes(BF16, M, d, 2048))
    buf = ws.buf
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tw.ffn_forward_q4(x, *q, workspace=ws)
    for k in range(3):
        call["product"]()
        x.copy_(_bf16(torch.Generator().manual_seed(70 + k), M, d))
        graph.replay()
        torch.cuda.synchronize()
        assert ws.buf is buf and torch.equal(out, tw.ffn_forward_q4(x, *q)), k
