"""examples/transformer_block.py with layer norm, the optimizer's step and low-rank adapters, whose calls are those of
a program, against the composition of the oracle's parts in fp64. Bounds as in test_gpu_block_example.py: each bf16 value
that is passed on is rounded once (2^-8 of it at most), so a chain of a few keeps a relative 2-norm error under 2^-6."""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

from synth import WORKLOADS, make_inputs, make_upstream_grad, scaled  # noqa: E402
from test_gpu_block_example import bits, ex, host, rel  # noqa: E402

tw = ex.tw
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def _training(M=96):
    w = scaled(WORKLOADS["tiny"], M=M)
    inp = make_inputs(w)
    rng = np.random.default_rng(4)

    def normal(*shape, at=0.0, scale=1.0):
        return torch.from_numpy((at + scale * rng.standard_normal(shape)).astype(np.float32))

    norm, bias = normal(w.d, at=1.0, scale=0.1).bfloat16().cuda(), normal(w.d, scale=0.1).bfloat16().cuda()
    layer = ex.TrainedLayer(norm, *(ex.to_device(b) for b in (inp.Wg, inp.WuT, inp.Wd)), w.T, w.C, 48, bias=bias)
    a, h = normal(w.M, w.d).cuda(), (normal(w.M, w.d) + 0.5).bfloat16().cuda()
    return w, inp, layer, a, h, ex.to_device(make_upstream_grad(w))


def test_train_step_with_layer_norm():
    w, inp, layer, a, h, dout = _training()
    p, seed, step = 0.2, 77, 3
    out, grads = ex.train_step(layer, a, h, dout, p, seed, step)
    da, dh, dnorm, dWg, dWuT, dWd, dbias = grads
    s = O.dropout(host(a), p, seed, 2 * step, host(h))
    n, mean, rstd = O.layernorm(s, host(layer.norm), host(layer.bias), ex.EPS)
    n_bits = bits(torch.from_numpy(n).bfloat16())
    y = O.dense_gated_ffn(n_bits, inp.Wg, inp.WuT, inp.Wd)
    assert rel(out, O.dropout(y, p, seed, 2 * step + 1, s)) < 2.0**-6
    dy = O.dropout(host(dout), p, seed, 2 * step + 1)
    dn, wWg, wWu, wWd = O.ffn_backward(n_bits, inp.Wg, inp.WuT, inp.Wd, bits(torch.from_numpy(dy).bfloat16()))
    ds, dw, db = O.layernorm_backward(dn, s, host(layer.norm), mean, rstd)
    ds = ds + host(dout)
    for name, got, want in (("dh", dh, ds), ("da", da, O.dropout(ds, p, seed, 2 * step)), ("dnorm", dnorm, dw), ("dbias", dbias, db),
                            ("dWg", dWg, wWg), ("dWuT", dWuT, wWu), ("dWd", dWd, wWd)):
        assert rel(got, want) < 2.0**-6, (name, rel(got, want))


@pytest.mark.parametrize("state_dtype", [F32, E4M3])
def test_update(state_dtype):
    """Two steps of the whole layer: the norm, the factor, and every weight; the layer's own bf16 tensors follow. A
    first step moves a weight by lr g / (|g| + eps), whatever its gradient's size: both steps' moves are compared, to
    2^-6 of them for fp32 states; 8-bit ones are off by a sixteenth in m and an eighth in sqrt(v) after the first step."""
    w, inp, layer, a, h, dout = _training()
    state = ex.optimizer_state(layer, state_dtype)
    start = [host(t.p) for t in state]
    m, v = [np.zeros_like(x) for x in start], [np.zeros_like(x) for x in start]
    want = [x.copy() for x in start]
    for step in (1, 2):
        _, grads = ex.train_step(layer, a, h, dout, 0.2, 77, step)
        g = [host(x) for x in grads[2:]]
        before = [x.copy() for x in want]
        clip = ex.update(state, grads[2:], step, 1e-2)
        norm = np.sqrt(sum((x * x).sum() for x in g))
        factor = min(1.0, 1.0 / norm)
        assert abs(clip[0].item() - norm) < 2.0**-20 * norm and abs(clip[1].item() - factor) < 2.0**-20 * factor
        for i, x in enumerate(g):
            want[i], m[i], v[i] = O.adamw(want[i], x, m[i], v[i], step, 1e-2, 0.9, 0.999, 1e-8, 0.1 if x.ndim > 1 else 0.0, factor)
            move, expected = host(state[i].p) - start[i], want[i] - start[i]
            off = np.linalg.norm(move - expected) / np.linalg.norm(expected)
            assert off < (2.0**-6 if state_dtype == F32 or step == 1 else 0.25), (i, step, off)
            assert torch.equal(state[i].copy, state[i].p.bfloat16()) and state[i].copy is layer.weights()[i]
            assert not np.array_equal(before[i], want[i])


def test_serve_with_adapters_from_a_graph():
    """Each replay reads the rows' adapters anew."""
    w = scaled(WORKLOADS["tiny"], M=5)
    rng = np.random.default_rng(6)
    inp = make_inputs(w)
    Wg, WuT, Wd = (ex.to_device(b) for b in (inp.Wg, inp.WuT, inp.Wd))
    norm = torch.ones(w.d, dtype=BF16, device="cuda")

    def normal(*shape, scale=1.0):
        return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda()

    adapters = tw.Adapters(normal(3, 8, w.d, scale=w.d**-0.5).bfloat16(), normal(3, w.d, 8).bfloat16(), normal(3).abs() + 0.5)
    layer = ex.ServedLayer.quantized(norm, Wg, WuT, Wd, adapters=adapters)
    plain = ex.ServedLayer.quantized(norm, Wg, WuT, Wd)
    index = torch.full((w.M,), -1, dtype=torch.int32, device="cuda")
    graph, y, h, out = ex.captured([layer], w.M, w.d, index)
    for rows in ([-1] * 5, [0, 0, 0, 0, 0], [2, 1, 0, -1, 2], [1, 7, 1, 2, -5]):
        y0, h0 = normal(w.M, w.d), normal(w.M, w.d).bfloat16()
        index.copy_(torch.tensor(rows, dtype=torch.int32))
        y.copy_(y0)
        h.copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        h1 = h0.clone()
        base = ex.serve([plain], y0, h1)
        r = tw.add_rmsnorm(y0, norm, ex.EPS, residual=h0, out_dtype=E4M3)
        x = host(r.n) * host(r.scale)[:, None]
        want = O.lora(x, np.array(rows), host(adapters.A), host(adapters.B), host(adapters.scaling), host(base))
        assert torch.equal(h, h1) and np.linalg.norm(host(out) - want) < 2.0**-20 * np.linalg.norm(want)


def test_the_program_runs(capsys):
    ex.main("all")
    said = capsys.readouterr().out
    assert "serve:" in said and "gradients' norm" in said and "nan" not in said
