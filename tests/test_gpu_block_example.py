"""examples/transformer_block.py, whose calls are those of a program, against the
composition of the oracle's parts in fp64.

Bounds: each bf16 value that is passed on is rounded once (2^-8 of it at most,
2^-9 on average), so a chain of a few such roundings keeps a relative 2-norm
error under 2^-6; sparse activity may differ where a gate is within rounding of
zero, whose terms are as small."""

from __future__ import annotations

import importlib.util
import os
import sys

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

from synth import WORKLOADS, make_inputs, make_upstream_grad, scaled  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("transformer_block", os.path.join(ROOT, "examples", "transformer_block.py"))
ex = importlib.util.module_from_spec(spec)
sys.modules[spec.name] = ex  # dataclasses look their module up
spec.loader.exec_module(ex)
tw = ex.tw


def host(t):
    return t.double().cpu().numpy()


def rel(got, want):
    return np.linalg.norm(host(got) - want) / np.linalg.norm(want)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def test_train_step():
    w = scaled(WORKLOADS["tiny"], M=96)
    inp = make_inputs(w)
    rng = np.random.default_rng(4)
    norm = torch.from_numpy((1 + 0.1 * rng.standard_normal(w.d)).astype(np.float32)).bfloat16().cuda()
    Wg, WuT, Wd = (ex.to_device(b) for b in (inp.Wg, inp.WuT, inp.Wd))
    layer = ex.TrainedLayer(norm, Wg, WuT, Wd, w.T, w.C, 48)
    a = torch.from_numpy(rng.standard_normal((w.M, w.d)).astype(np.float32)).cuda()
    h = torch.from_numpy(rng.standard_normal((w.M, w.d)).astype(np.float32)).bfloat16().cuda()
    dout = ex.to_device(make_upstream_grad(w))
    p, seed, step = 0.2, 77, 3
    out, (da, dh, dnorm, dWg, dWuT, dWd) = ex.train_step(layer, a, h, dout, p, seed, step)
    again = ex.train_step(layer, a, h, dout, p, seed, step)
    assert torch.equal(out, again[0]) and all(torch.equal(x, y) for x, y in zip((da, dh, dnorm), again[1][:3]))

    s = O.dropout(host(a), p, seed, 2 * step, host(h))
    n, rstd = O.rmsnorm(s, host(norm), ex.EPS)
    n_bits = bits(torch.from_numpy(n).bfloat16())
    y = O.dense_gated_ffn(n_bits, inp.Wg, inp.WuT, inp.Wd)
    want_out = O.dropout(y, p, seed, 2 * step + 1, s)
    assert rel(out, want_out) < 2.0**-6
    dy = O.dropout(host(dout), p, seed, 2 * step + 1)
    dn, wWg, wWu, wWd = O.ffn_backward(n_bits, inp.Wg, inp.WuT, inp.Wd, bits(torch.from_numpy(dy).bfloat16()))
    ds, dw = O.rmsnorm_backward(dn, s, host(norm), rstd)
    ds = ds + host(dout)
    for name, got, want in (("dh", dh, ds), ("da", da, O.dropout(ds, p, seed, 2 * step)), ("dnorm", dnorm, dw),
                            ("dWg", dWg, wWg), ("dWuT", dWuT, wWu), ("dWd", dWd, wWd)):
        assert rel(got, want) < 2.0**-6, (name, rel(got, want))


def test_serve_graph():
    w = scaled(WORKLOADS["tiny"], M=3)
    rng = np.random.default_rng(6)
    layers, weights = [], []
    for i in range(2):
        inp = make_inputs(w, seed=50 + i)
        norm = torch.from_numpy((1 + 0.1 * rng.standard_normal(w.d)).astype(np.float32)).bfloat16().cuda()
        layers.append(ex.ServedLayer.quantized(norm, *(ex.to_device(b) for b in (inp.Wg, inp.WuT, inp.Wd)), group=64))
        parts = (O.decode_bf16(inp.Wg), O.decode_bf16(inp.WuT), O.decode_bf16(inp.Wd).T)
        weights.append((host(norm), [O.q4_dequantize(*O.q4_quantize(m, 64), None, 64) for m in parts]))
    graph, y_in, h, out = ex.captured(layers, w.M, w.d)
    e4m3 = torch.float8_e4m3fn
    for token in range(4):
        x = torch.from_numpy(rng.standard_normal((w.M, w.d)).astype(np.float32)).cuda()
        start = torch.from_numpy(rng.standard_normal((w.M, w.d)).astype(np.float32)).bfloat16().cuda()
        y_in.copy_(x)
        h.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        h2 = start.clone()
        eager = ex.serve(layers, x, h2)
        assert torch.equal(out, eager) and torch.equal(h, h2), token

        y, s = host(x), host(start)
        for norm, (Wg, Wu, Wd) in weights:
            s = s + y
            n, _ = O.rmsnorm(s, norm, ex.EPS)
            scale = np.abs(n).max(axis=1, keepdims=True) / 448
            q = torch.from_numpy(n / scale).float().to(e4m3).double().numpy() * scale
            s = torch.from_numpy(s).bfloat16().double().numpy()
            y = O.gated_hidden(q, Wg, Wu) @ Wd.T
        # where a value lies within fp32 rounding of two e4m3 values the step is 2^-4 of it: a
        # few of them in a row of 256 move y by less than 2^-4 of its norm
        assert rel(out, y) < 2.0**-4, (token, rel(out, y))
