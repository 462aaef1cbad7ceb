"""The gradients' norm and the optimizer's step on the GPU, through the binding, against the fp64 oracle.

Error bounds, u = 2^-24, from the arithmetic (constants are rounded to fp32: u each):
* g' = s g: u. m = b1 m + (1 - b1) g': 5 u of the sum of magnitudes. v, all of it positive:
  7 u of itself, its root 5 u (half of that, the root's own rounding, and slack).
* the update rate m / (root k + eps): m's error over the denominator, and 16 u of itself; p: 2 u
  of the magnitudes of p and of what is taken away.
* 8-bit states: what is kept is the oracle's rounding of a value as far off as the unrounded m or
  root is, plus 4 u for the scale; the rounding never falls as the value rises, so the code lies between those
  of the two ends.
* the norm: squares are exact in fp64, sums off by 2^-40 at most, one rounding to fp32."""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402

DEV = torch.device("cuda", 0)
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0**-24
SEED, OFFSET = 0x123456789ABCDEF0, (7 << 32) + 3
TINY = 2.0**-148  # two steps under 2^-126


def host(t):
    return t.double().cpu().numpy().reshape(-1)


def rand(rng, n, dtype=F32, scale=1.0):
    return torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)).to(dtype).to(DEV)


def odd(t):
    """The same values one element past an aligned address."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    flat[1:].view(torch.uint8 if t.dtype == E4M3 else t.dtype).copy_(t.flatten().view(torch.uint8 if t.dtype == E4M3 else t.dtype))
    return flat[1:].view(t.shape)


def state_of(rng, n, dtype, scale):
    """(p, m, v as the step meets them, AdamTensors): a state that earlier steps have left."""
    p, m, root = rand(rng, n), rand(rng, n, scale=scale), rand(rng, n, scale=scale).abs()
    if n > 40:
        m[::7], root[::11] = 0, 0
    if dtype == F32:
        return tw.AdamTensors(p, m, root.square())
    made = []
    for v in (m, root):
        s = O.block_scales(host(v)).astype(np.float32)
        q = O.to_neighbour(np.clip(host(v) / s.astype(np.float64)[np.arange(n) // 256], -448, 448), np.full(n, 127))
        made += [torch.from_numpy(q.astype(np.float32)).to(DEV).to(E4M3), torch.from_numpy(s).to(DEV)]
    return tw.AdamTensors(p, made[0], made[2], made[1], made[3])


def values(t):
    """p, m, v of an AdamTensors in fp64."""
    p, m, v = host(t.p), host(t.m.float()), host(t.v.float())
    if t.m_scale is not None:
        at = np.arange(len(p)) // 256
        m[~np.isfinite(host(t.m_scale)[at])], v[~np.isfinite(host(t.v_scale)[at])] = np.nan, np.nan
        m, v = m * host(t.m_scale)[at], (v * host(t.v_scale)[at]) ** 2
    return p, m, v


def close(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}")


def check(before, g, after, number, step, lr, betas, eps, decay, scale, seed, offset, copy):
    p0, m0, v0 = before
    b1, b2 = betas
    gs = g * scale
    p, m, v = O.adamw(p0, g, m0, v0, step, lr, b1, b2, eps, decay, scale)
    e_m = 5 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * gs)) + TINY
    e_v = 7 * U * v + TINY
    root = np.sqrt(v)
    e_root = np.where(v > 2.0**-120, 5 * U * root, np.sqrt(2 * TINY) + 5 * U * root)
    k = 1 / np.sqrt(1 - b2**step)
    rate = lr / (1 - b1**step)
    low = np.maximum((root - e_root) * k, 0) + eps
    hat = rate * np.abs(m) / (root * k + eps)
    e_hat = rate * e_m / low + hat * (16 * U + e_root * k / low)
    near = 2 * U * (np.abs(p0) + np.abs(p) + np.abs(lr * decay * p0) + hat) + e_hat + TINY
    close(host(after.p), p, near, f"p of tensor {number}")
    if copy is not None:
        assert torch.equal(copy.flatten(), after.p.flatten().to(BF16)), number
    if after.m_scale is None:
        close(host(after.m), m, e_m, f"m of tensor {number}")
        close(host(after.v), v, e_v, f"v of tensor {number}")
        return
    n = len(p)
    at = np.arange(n) // 256
    bits = O.state_bits(n, number, seed, offset)
    for name, x, e, codes, scales, draw, least in (("m", m, e_m, after.m, after.m_scale, bits & 255, 0.0),
                                                   ("root", root, e_root, after.v, after.v_scale, bits >> 8, 2.0**-9)):
        want = O.block_scales(x)
        e_scale = O.block_scales(np.abs(x) + e) - want + 2 * U * want
        close(host(scales), want, e_scale, f"{name}'s scales of tensor {number}")
        s = host(scales)[at]  # the kernel's own: x / s is what its rounding meets
        q, off = x / s, e / s + 4 * U * np.abs(x / s)
        lo, hi = O.to_neighbour(np.clip(q - off, -448, 448), draw), O.to_neighbour(np.clip(q + off, -448, 448), draw)
        if least:  # the root: at least one step, unless it may be zero
            lo = np.where(x - e > 0, np.maximum(lo, least), np.maximum(lo, 0))
            hi = np.maximum(hi, least) * (x + e > 0)
        got = host(codes.float())
        bad = ~((got >= lo) & (got <= hi))
        assert not bad.any(), (name, number, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], lo[bad][:3], hi[bad][:3])


# one element, both sides of a block, of a chunk and of a cut group of 8
NUMELS = [1, 255, 256, 257, 7, 8, 9, 2047, 2048, 2049, 5000]


@pytest.mark.parametrize("state", [F32, E4M3])
@pytest.mark.parametrize("step,decay,scale,copies,place", [(1, 0.0, None, False, "in place"), (7, 0.1, 0.37, True, "elsewhere"),
                                                           (100000, 0.5, 3.0, True, "odd")])
def test_adamw_step(state, step, decay, scale, copies, place):
    print(f"[adamw] {state} step {step} {place}", flush=True)
    rng = np.random.default_rng(step)
    hyper = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8)
    tensors = [tw.AdamTensors.zero(rand(rng, n), state) if step == 1 else state_of(rng, n, state, 10.0 ** -(i % 5))
               for i, n in enumerate(NUMELS)]
    grads = [rand(rng, n, BF16 if i % 3 == 1 else F32, 10.0 ** -(i % 5)) for i, n in enumerate(NUMELS)]
    if place == "odd":
        tensors = [tw.AdamTensors(*(odd(t) for t in (a.p, a.m, a.v)),
                                  *(None if s is None else odd(s) for s in (a.m_scale, a.v_scale))) for a in tensors]
        grads = [odd(g) for g in grads]
    out = [tw.AdamTensors.zero(torch.full_like(t.p, 9.0), state) for t in tensors] if place == "elsewhere" else None
    to = out or tensors
    for t in to if copies else []:
        t.copy = torch.zeros_like(t.p, dtype=BF16)
    before = [values(t) for t in tensors]
    kept = [t.p.clone() for t in tensors]
    tw.adamw_step(tensors, grads, step, weight_decay=decay, seed=SEED, offset=OFFSET, out=out,
                  grad_scale=None if scale is None else torch.full((1,), scale, device=DEV), **hyper)
    for i, (b, g, t) in enumerate(zip(before, grads, to)):
        check(b, host(g.float()), t, i, step, hyper["lr"], hyper["betas"], hyper["eps"], decay,
              1.0 if scale is None else float(np.float32(scale)), SEED, OFFSET, t.copy)
        assert out is None or torch.equal(kept[i], tensors[i].p)


@pytest.mark.parametrize("state", [F32, E4M3])
def test_more_tensors_than_a_launch_takes(state):
    """70 tensors, empty ones among them, of one and of two dimensions, a weight decay each."""
    print(f"[adamw] 70 tensors {state}", flush=True)
    rng = np.random.default_rng(5)
    sizes = [0 if i % 9 == 4 else int(rng.integers(1, 3000)) for i in range(70)]
    sizes[31], sizes[63], sizes[69] = 0, 0, 0  # a launch's last
    tensors = [state_of(rng, n, state, 1e-2) if n else tw.AdamTensors.zero(torch.empty(0, device=DEV), state) for n in sizes]
    grads = [rand(rng, n, scale=1e-2) for n in sizes]
    for i, n in enumerate(sizes):
        if n % 2 == 0 and n:
            t = tensors[i]
            t.p, t.m, t.v, grads[i] = t.p.view(2, -1), t.m.view(2, -1), t.v.view(2, -1), grads[i].view(2, -1)
    before = [values(t) for t in tensors]
    decay = [0.01 * i for i in range(70)]
    tw.adamw_step(tensors, grads, 3, 1e-3, weight_decay=decay, seed=SEED, offset=OFFSET)
    for i, n in enumerate(sizes):
        if n:
            check(before[i], host(grads[i]), tensors[i], i, 3, 1e-3, (0.9, 0.999), 1e-8, decay[i], 1.0, SEED, OFFSET, None)


@pytest.mark.parametrize("state", [F32, E4M3])
def test_nothing_beside_the_tensors_is_written(state):
    rng = np.random.default_rng(6)
    for n in (1, 300, 2049, 4096):
        kinds = {}
        for k, t in (("p", F32), ("m", state), ("v", state), ("copy", BF16)):
            whole = torch.full((n + 512,), 7, dtype=torch.uint8, device=DEV).to(F32).to(t) if t != E4M3 else torch.full(
                (n + 512,), 0x40, dtype=torch.uint8, device=DEV).view(E4M3)
            kinds[k] = whole
        scales = {k: torch.full((-(-n // 256) + 8,), 7.0, device=DEV) for k in ("m_scale", "v_scale")} if state == E4M3 else {}
        inner = {k: t[256:256 + n] for k, t in kinds.items()} | {k: s[4:-4] for k, s in scales.items()}
        before = {k: t.clone() for k, t in (kinds | scales).items()}
        tw.adamw_step([tw.AdamTensors(**inner)], [rand(rng, n)], 2, 1e-3)
        for k, t in (kinds | scales).items():
            edge = 256 if k in kinds else 4
            raw = (lambda a: a.view(torch.uint8)) if t.dtype == E4M3 else (lambda a: a)
            assert torch.equal(raw(t)[:edge], raw(before[k])[:edge]) and torch.equal(raw(t)[-edge:], raw(before[k])[-edge:]), k
            # (a step of 1e-3 at most moves no 7 in bf16, whose steps there are 2^-6)
            assert k == "copy" or not torch.equal(raw(t), raw(before[k])), k
        assert torch.equal(inner["copy"], inner["p"].to(BF16))


def bytes_of(t):
    return [x.flatten().view(torch.uint8).clone() for x in (t.p, t.m, t.v, t.m_scale, t.v_scale, t.copy) if x is not None]


@pytest.mark.parametrize("state", [F32, E4M3])
def test_skipped_steps_and_values_that_are_not_finite(state):
    rng = np.random.default_rng(7)
    t = state_of(rng, 1000, state, 1e-2)
    t.copy = torch.ones(1000, dtype=BF16, device=DEV)
    g = rand(rng, 1000)
    before = bytes_of(t)
    for bad in (0.0, float("nan"), float("inf"), float("-inf")):
        tw.adamw_step([t], [g], 2, 1e-2, grad_scale=torch.full((1,), bad, device=DEV))
        assert all(torch.equal(a, b) for a, b in zip(before, bytes_of(t))), bad
    # what grad_norm leaves for a gradient that is not finite skips the step, with no wait between
    for bad in (float("nan"), float("inf")):
        h = g.clone()
        h[700] = bad
        norm = tw.grad_norm([h], 1.0)
        tw.adamw_step([t], [h], 2, 1e-2, grad_scale=norm[1:])
        assert not torch.isfinite(norm[0]) and all(torch.equal(a, b) for a, b in zip(before, bytes_of(t))), bad
        # without it: that element, or in 8 bits its block's states, from then on
        u = tw.AdamTensors(t.p.clone(), t.m.clone(), t.v.clone(), *(None if s is None else s.clone() for s in (t.m_scale, t.v_scale)))
        tw.adamw_step([u], [h], 2, 1e-2)
        p, m, v = values(u)
        at = np.arange(1000)
        assert np.array_equal(~np.isfinite(p), at == 700)
        lost = (at == 700) if state == F32 else (at // 256 == 700 // 256)
        assert np.array_equal(~np.isfinite(m), lost) and np.array_equal(~np.isfinite(v), lost)
    with pytest.raises(ValueError):
        tw.adamw_step([t], [g], 2, 1e-2, grad_scale=torch.ones(2, device=DEV))


def test_small_and_large_gradients():
    """Squares that leave the range: v of 2^-149 and below is zero or a step, g' of 2^64 and above an
    infinite v, which moves nothing."""
    g = torch.tensor([1e-30, 1e-20, 1e-12, 1.0, 1e18, 1e25, 3e38], device=DEV)
    for state in (F32, E4M3):
        for i in range(7):
            t = tw.AdamTensors.zero(torch.ones(1, device=DEV), state)
            tw.adamw_step([t], [g[i:i + 1]], 1, 0.5)
            moved = 1 - t.p.item()
            if i in (2, 3, 4):
                x = float(g[i])
                assert abs(moved - 0.5 * x / (x + 1e-8)) < 2.0**-18
            elif i < 2:
                assert 0 <= moved <= 0.5 * 1e-20 / 1e-8 + 2.0**-24
            else:
                assert moved == 0


def test_steps_in_8_bits_follow_those_in_32():
    """A decay of a thousandth a step is far below half a step of e4m3: the second moment follows all the same.
    A root moves by draws of one part in 8 to 16 with that mean; after 3000 steps from 1 to 1/10 of
    the gradients, the means over 4096 elements are within a tenth."""
    g = torch.Generator(device=DEV).manual_seed(3)
    n = 4096
    a, b = tw.AdamTensors.zero(torch.zeros(n, device=DEV)), tw.AdamTensors.zero(torch.zeros(n, device=DEV), E4M3)
    for step in range(1, 3201):
        grad = torch.randn(n, generator=g, device=DEV) * (1.0 if step <= 200 else 0.1)
        for t in (a, b):
            tw.adamw_step([t], [grad], step, 1e-3, seed=1, offset=step)
    v32, v8 = values(a)[2].mean(), values(b)[2].mean()
    # v32 is near 0.01 + 0.18 exp(-3): 8 bits to nearest would have stayed at 0.18
    assert v32 < 0.03 and 0.9 * v32 < v8 < 1.25 * v32
    m32, m8 = values(a)[1], values(b)[1]
    assert np.linalg.norm(m8 - m32) < 0.15 * np.linalg.norm(m32)


@pytest.mark.parametrize("sizes,types", [([1], [F32]), ([5000], [BF16]), ([8191, 8192, 8193, 1, 0, 77], [F32, BF16] * 3),
                                         ([1000] * 70, [F32] * 70), ([3_000_001], [F32])])
@pytest.mark.parametrize("max_norm", [1.0, 1e9, float("inf")])
def test_grad_norm(sizes, types, max_norm):
    rng = np.random.default_rng(len(sizes))
    grads = [rand(rng, n, t, 10.0 ** -(i % 3)) for i, (n, t) in enumerate(zip(sizes, types))]
    if len(sizes) == 6:
        grads = [odd(g) for g in grads]
    out = tw.grad_norm(grads, max_norm)
    want = np.sqrt(sum((host(g) ** 2).sum() for g in grads))
    got = host(out)
    assert abs(got[0] - want) <= U * want * (1 + 2.0**-10)
    factor = min(1.0, max_norm / want)
    assert abs(got[1] - factor) <= U * factor * (1 + 2.0**-10) and got[1] <= 1
    assert torch.equal(out, tw.grad_norm(grads, max_norm))


def test_grad_norm_over_the_range():
    z = torch.zeros(100, device=DEV)
    assert tw.grad_norm([z], 1.0).tolist() == [0.0, 1.0]
    assert tw.grad_norm([torch.empty(0, device=DEV)], 1.0).tolist() == [0.0, 1.0]
    big = torch.full((100,), 1e30, device=DEV)  # squares past fp32's range
    out = host(tw.grad_norm([big], 1.0))
    assert abs(out[0] / (10 * float(np.float32(1e30))) - 1) < 2 * U and abs(out[1] * out[0] - 1) < 4 * U
    small = torch.full((100,), 2.0**-140, device=DEV)
    assert tw.grad_norm([small], 1.0).tolist() == [10 * 2.0**-140, 1.0]
    for bad in (float("nan"), float("inf"), float("-inf")):
        x = torch.ones(20000, device=DEV)
        x[19999] = bad
        norm, factor = tw.grad_norm([z, x], 1.0).tolist()
        assert not np.isfinite(norm) and (factor == 0 or np.isnan(factor)), bad
        norm, factor = tw.grad_norm([z, x]).tolist()
        assert not np.isfinite(norm) and (factor == 0 or np.isnan(factor)), bad
    with pytest.raises(tw.TwellError):
        tw.grad_norm([z], 0.0)
    with pytest.raises(ValueError):
        tw.grad_norm([z[::2]], 1.0)
    with pytest.raises(TypeError):
        tw.grad_norm([z.half()], 1.0)


@pytest.mark.parametrize("state", [F32, E4M3])
def test_captured_and_replayed(state):
    """Norm, clipping and step in a graph, replayed with eager work between, against eager calls."""
    rng = np.random.default_rng(9)
    sizes = [4000, 300, 70000]
    kept = [tw.AdamTensors.zero(rand(rng, n), state, copy=torch.zeros(n, dtype=BF16, device=DEV)) for n in sizes]
    eager = [tw.AdamTensors(*(None if x is None else x.clone() for x in (t.p, t.m, t.v, t.m_scale, t.v_scale, t.copy)))
             for t in kept]
    grads = [rand(rng, n) for n in sizes]

    def step(tensors):
        norm = tw.grad_norm(grads, 1.0)
        tw.adamw_step(tensors, grads, 5, 1e-2, grad_scale=norm[1:], seed=3, offset=5)
        return norm

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # a first call outside the capture loads the kernels
        step([tw.AdamTensors.zero(torch.zeros(n, device=DEV), state) for n in sizes])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step(kept)
    for k in range(4):
        for g in grads:
            g.copy_(rand(rng, g.numel()))
        want = step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want), k
        for a, b in zip(kept, eager):
            assert all(torch.equal(x, y) for x, y in zip(bytes_of(a), bytes_of(b))), k


def test_norms_on_two_streams_at_once():
    rng = np.random.default_rng(10)
    lists = [[rand(rng, 400000)], [rand(rng, 900000), rand(rng, 77)]]
    want = [tw.grad_norm(g, 1.0) for g in lists]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for s, g, o in zip(streams, lists, got):
            with torch.cuda.stream(s):
                o.append(tw.grad_norm(g, 1.0))
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(x, w) for x in o)


def test_a_long_tensor():
    """Offsets past 32 bits: elements around 2^32 of a tensor in 8 bits, against the same ones on their own
    where only the place in the tensor differs (the draws do: with representable values they change nothing)."""
    n = (1 << 32) + 777
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < 80 << 30:
        pytest.skip("needs 80 GiB of device memory")
    print(f"[adamw] {n} elements", flush=True)
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, device=DEV, dtype=BF16)
    t = tw.AdamTensors.zero(p, E4M3)
    # 448 and 2^k steps of a block: exact in e4m3
    at = [0, 255, (1 << 31) - 256, (1 << 31) + 3, (1 << 32) - 1, 1 << 32, n - 1]
    for i in at:
        g[i] = 1.0
    tw.adamw_step([t], [g], 1, 0.5, betas=(0.5, 0.75), eps=0.0)
    for i in at:
        assert p[i].item() == -0.5, i
        block = i // 256
        assert abs(t.m[i].float().item() * t.m_scale[block].item() - 0.5) < 2.0**-20
        assert abs(t.v[i].float().item() * t.v_scale[block].item() - 0.5) < 2.0**-20
    norm = tw.grad_norm([g], 1.0)
    assert norm[0].item() == np.float32(np.sqrt(len(at)))
    del p, g, t
    torch.cuda.empty_cache()
