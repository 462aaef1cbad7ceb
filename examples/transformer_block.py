"""The FFN half of a transformer block with everything around it on the library's
kernels, as a program uses them:

* serving: residual addition and RMS norm in one call with 8-bit output, then the
  layer with 4-bit weights on that output, layer after layer, captured in a HIP
  graph and replayed a token at a time;
* training: dropout, residual addition and norm, the sparse FFN, dropout into the
  residual stream again, and the backward of all of it.

Run: python examples/transformer_block.py [serve|train]   (needs the GPU)
"""

from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from synth import WORKLOADS, make_inputs, make_upstream_grad, scaled  # noqa: E402

EPS = 1e-6


def to_device(bits, device="cuda"):
    import numpy as np

    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(torch.bfloat16)


# ------------------------------------------------------------------ serving
@dataclass
class ServedLayer:
    norm: torch.Tensor  # bf16 [d]
    Wg: tw.Q4  # [F, d]
    Wu: tw.Q4  # [F, d]
    Wd: tw.Q4  # [d, F]: down_proj.weight itself

    @classmethod
    def quantized(cls, norm, Wg, WuT, Wd, group=128):
        """From the bf16 layer as the other calls take it (Wd [F, d])."""
        return cls(norm, tw.q4_quantize(Wg, group), tw.q4_quantize(WuT, group),
                   tw.q4_quantize(Wd.t().contiguous(), group))


def serve(layers, y, h):
    """y float32 [M, d] joins the residual stream h (bf16, updated in place)
    before each layer; returns the last layer's y."""
    for layer in layers:
        r = tw.add_rmsnorm(y, layer.norm, EPS, residual=h, out_dtype=torch.float8_e4m3fn, h=h)
        y = tw.ffn_forward_q4(r.n, layer.Wg, layer.Wu, layer.Wd, x_scale=r.scale)
    return y


def captured(layers, M, d):
    """serve() of M rows as a graph: (graph, y in, h, y out). The calls' scratch is
    allocated in the capture, so it is the graph's own."""
    y, h = torch.zeros(M, d, device="cuda"), torch.zeros(M, d, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a first call outside the capture loads the kernels
        serve(layers, y, h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = serve(layers, y, h)
    return graph, y, h, out


# ------------------------------------------------------------------ training
@dataclass
class TrainedLayer:
    norm: torch.Tensor  # bf16 [d]
    Wg: torch.Tensor  # bf16 [F, d], as are the next two
    WuT: torch.Tensor
    Wd: torch.Tensor
    T: int
    C: int
    K: int  # width of the hybrid format's block


def train_step(layer, a, h, dout, p, seed, step):
    """One layer's forward and backward. a (float32: what the branch before
    gives) and h (bf16: the residual stream) come in,
        s = h + dropout(a),  n = norm(s),  y = FFN(n),  out = s + dropout(y),
    dout is the gradient of out. Returns out, and the gradients (da bf16, dh bf16,
    dnorm, dWg, dWuT, dWd)."""
    drop_a, drop_y = dict(p=p, seed=seed, offset=2 * step), dict(p=p, seed=seed, offset=2 * step + 1)
    M, F = a.shape[0], layer.Wg.shape[0]
    r = tw.add_rmsnorm(a, layer.norm, EPS, residual=h, **drop_a)
    packed, spill = tw.gate_pack_spill(r.n, layer.Wg, layer.T, layer.C, M * (F // layer.T))
    hybrid = tw.hybrid_pack(packed, F, layer.K, M, spill=spill)
    y = tw.ffn_forward(r.n, layer.Wg, layer.WuT, layer.Wd, layer.T, layer.C)
    out = tw.dropout(y, residual=r.h, **drop_y)

    dy = tw.dropout(dout, out_dtype=torch.bfloat16, **drop_y)
    dn, dWg, dWuT, dWd = tw.ffn_backward(r.n, layer.Wg, layer.WuT, layer.Wd, dy, hybrid)
    dh, da, dnorm = tw.add_rmsnorm_backward(dn, r.h, layer.norm, r.rstd, dh=dout, dx_dtype=torch.bfloat16, **drop_a)
    return out, (da, dh, dnorm, dWg, dWuT, dWd)


def _layers(w, n):
    """n synthetic layers of a workload's shape: (norm, Wg, WuT, Wd) each."""
    g = torch.Generator().manual_seed(1)
    for i in range(n):
        inp = make_inputs(w, seed=w.seed + i)
        norm = (1 + 0.1 * torch.randn(w.d, generator=g)).bfloat16().cuda()
        yield (norm, *(to_device(b) for b in (inp.Wg, inp.WuT, inp.Wd)))


def main(what="all"):
    if what in ("all", "serve"):
        w = scaled(WORKLOADS["decode_m1"], M=4)
        layers = [ServedLayer.quantized(*parts) for parts in _layers(w, 2)]
        graph, y, h, out = captured(layers, w.M, w.d)
        for token in range(4):
            y.copy_(torch.randn(w.M, w.d, generator=torch.Generator().manual_seed(token)))
            h.zero_()
            graph.replay()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(50):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"serve: {w.M} rows, {len(layers)} layers d={w.d} F={w.F} in 4 bits: "
              f"{begin.elapsed_time(end) / 50 / len(layers) * 1e3:.1f} us a layer, |y| {out.norm().item():.3f}")
    if what in ("all", "train"):
        w = scaled(WORKLOADS["ffn1p5b"], M=512)
        norm, Wg, WuT, Wd = next(iter(_layers(w, 1)))
        layer = TrainedLayer(norm, Wg, WuT, Wd, w.T, w.C, 128)
        a = torch.randn(w.M, w.d, generator=torch.Generator().manual_seed(5)).cuda()
        h = torch.randn(w.M, w.d, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
        dout = to_device(make_upstream_grad(w))
        for step in range(2):
            out, grads = train_step(layer, a, h, dout, 0.1, 1234, step)
        torch.cuda.synchronize()
        names = ("da", "dh", "dnorm", "dWg", "dWuT", "dWd")
        print(f"train: {w.M} rows, |out| {out.float().norm().item():.3f}, " +
              ", ".join(f"|{n}| {g.float().norm().item():.3g}" for n, g in zip(names, grads)))


if __name__ == "__main__":
    main(*sys.argv[1:2])
