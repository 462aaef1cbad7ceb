"""The optimizer's step where its coefficients matter: many steps, coefficients at both ends, values at the ends of the
range; and the draws of 8-bit states by default."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_adamw import DEV, E4M3, F32, U, bytes_of, check, host, rand, state_of, values  # noqa: E402


def test_second_moments_over_many_steps_have_no_bias():
    """20000 steps with c = 1 - beta2 = 1e-4 and g^2 uniform over [0, 2] against fp64, in the mean over 2^16 elements. c g^2
    is uniform over W = 1680 ulps of v (which stays near 1; an ulp is up to 2 U of it), so that whatever v is, a step's
    rounding has a mean of at most 1 / (8 W) ulp (what a cut period leaves), 1.5e-4 U: 1.3 U over the sum of 0.9999^k = 8647 steps.
    Its chance, at most U / sqrt(3) a step: times sqrt(1 / 2c) = 71, over 256 for the mean, six deviations: U. What c g^2
    and its sum with the small part of v are rounded by: 3 U of c, for v all of c's 1 / c steps, 3 U. The rounding of c moves
    both ends of an average alike: 2 U. 8 U in all; a coefficient of v off by 1.66e-8 is 2400 U."""
    print("[adamw] many steps", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(4)
    n, beta2 = 1 << 16, 0.9999
    t = tw.AdamTensors(torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), torch.ones(n, device=DEV))
    v = torch.ones(n, device=DEV, dtype=torch.float64)
    for step in range(1, 20001):
        g = torch.rand(n, generator=gen, device=DEV).mul_(2).sqrt_()
        tw.adamw_step([t], [g], step, 0.0, betas=(0.9, beta2))
        v.lerp_(g.double().square_(), 1.0 - beta2)
    off = (t.v.double() / v - 1).mean().item()
    assert abs(off) < 8 * U, off / U


@pytest.mark.parametrize("state", [F32, E4M3])
@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.3, 0.25), (0.5, 0.5), (0.51, 0.49), (0.75, 0.9999999), (1 - 2.0**-53, 1 - 2.0**-53)])
def test_coefficients(state, betas):
    """Against the formula, with old moments far larger and far smaller than the gradient."""
    print(f"[adamw] {state} {betas}", flush=True)
    rng = np.random.default_rng(2)
    n = 3000
    for size, of_state in ((1.0, 1.0), (1e-5, 1.0), (1.0, 1e-5)):
        t = state_of(rng, n, state, of_state)
        g = rand(rng, n, scale=size)
        before = values(t)
        tw.adamw_step([t], [g], 4, 1e-2, betas=betas, seed=5, offset=6)
        check(before, host(g), t, 0, 4, 1e-2, betas, 1e-8, 0.0, 1.0, 5, 6, None)


def test_moments_at_the_ends_of_the_range():
    """The old moment and the gradient further apart than the largest fp32, and squares past it: v is infinite from then
    on, and moves nothing."""
    big = 3e38
    for beta1 in (0.9, 0.3):
        m0, g = torch.tensor([big, -big, big, 0.0, 1.0], device=DEV), torch.tensor([-big, big, big, big, -1.0], device=DEV)
        t = tw.AdamTensors(torch.ones(5, device=DEV), m0.clone(), torch.zeros(5, device=DEV))
        tw.adamw_step([t], [g], 3, 0.1, betas=(beta1, 0.999))
        want = beta1 * host(m0) + (1 - beta1) * host(g)
        assert (np.abs(host(t.m) - want) <= 5 * U * (beta1 * np.abs(host(m0)) + (1 - beta1) * np.abs(host(g)))).all()
        assert torch.isinf(t.v[:4]).all() and (t.p[:4] == 1).all() and torch.isfinite(t.v[4])
        for step in (4, 5):  # small gradients again: still infinite, not NaN
            tw.adamw_step([t], [torch.ones(5, device=DEV)], step, 0.1, betas=(beta1, 0.999))
            assert torch.isinf(t.v[:4]).all() and (t.v[:4] > 0).all() and torch.isfinite(t.m).all() and (t.p[:4] == 1).all()
    for beta2 in (0.999, 0.3):
        t = tw.AdamTensors.zero(torch.ones(3, device=DEV))
        tw.adamw_step([t], [torch.tensor([float("nan"), 1e25, 1.0], device=DEV)], 1, 0.5, betas=(0.9, beta2))
        assert t.v.isnan().tolist() == [True, False, False] and t.v.isinf().tolist() == [False, True, False]


def test_offset_by_default_is_the_step():
    """Each step of 8-bit states has draws of its own; a given offset, 0 too, is taken as it is."""
    rng = np.random.default_rng(3)
    kept = state_of(rng, 5000, E4M3, 1e-2)
    g = rand(rng, 5000, scale=1e-2)

    def after(step, **kw):
        t = tw.AdamTensors(*(x.clone() for x in (kept.p, kept.m, kept.v, kept.m_scale, kept.v_scale)))
        tw.adamw_step([t], [g], step, 1e-3, seed=9, **kw)
        return bytes_of(t)[1:]

    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert same(after(7), after(7, offset=7)) and not same(after(7), after(7, offset=0))
    assert same(after(8), after(8, offset=8)) and not same(after(8), after(8, offset=7))


def test_steps_in_8_bits_with_offsets_by_default():
    """As test_steps_in_8_bits_follow_those_in_32, whose bounds these are, without an offset: with one draw for all
    steps most roots would not fall at all."""
    g = torch.Generator(device=DEV).manual_seed(3)
    n = 4096
    a, b = tw.AdamTensors.zero(torch.zeros(n, device=DEV)), tw.AdamTensors.zero(torch.zeros(n, device=DEV), E4M3)
    for step in range(1, 3201):
        grad = torch.randn(n, generator=g, device=DEV) * (1.0 if step <= 200 else 0.1)
        for t in (a, b):
            tw.adamw_step([t], [grad], step, 1e-3, seed=1)
    v32, v8 = values(a)[2].mean(), values(b)[2].mean()
    assert v32 < 0.03 and 0.9 * v32 < v8 < 1.25 * v32
    m32, m8 = values(a)[1], values(b)[1]
    assert np.linalg.norm(m8 - m32) < 0.15 * np.linalg.norm(m32)


@pytest.mark.parametrize("state", [F32, E4M3])
def test_tensors_of_one_buffer(state):
    """Views that touch are tensors like any others, in place and into another buffer; views that share an element are
    refused, whichever comes first."""
    print(f"[adamw] one buffer {state}", flush=True)
    rng = np.random.default_rng(6)
    sizes = [1000, 777, 1, 4096]
    blocks = [-(-n // 256) for n in sizes]

    def packed(tensors):
        """The same tensors, each kind in one buffer without gaps."""
        def pack(k, n):
            parts = [getattr(t, k) for t in tensors]
            if parts[0] is None:
                return parts
            raw = torch.uint8 if parts[0].dtype == E4M3 else parts[0].dtype
            return torch.cat([x.view(raw) for x in parts]).view(parts[0].dtype).split(n)

        kinds = {k: pack(k, blocks if "scale" in k else sizes) for k in ("p", "m", "v", "m_scale", "v_scale", "copy")}
        return [tw.AdamTensors(*(kinds[k][i] for k in ("p", "m", "v", "m_scale", "v_scale", "copy"))) for i in range(len(sizes))]

    alone = [state_of(rng, n, state, 1e-2) for n in sizes]
    for t, n in zip(alone, sizes):
        t.copy = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    grads = [rand(rng, n, scale=1e-2) for n in sizes]
    together, out = packed(alone), packed([tw.AdamTensors.zero(t.p, state, copy=t.copy) for t in alone])
    tw.adamw_step(together, grads, 3, 1e-2, seed=1, out=out)
    tw.adamw_step(alone, grads, 3, 1e-2, seed=1)
    tw.adamw_step(together, grads, 3, 1e-2, seed=1)
    for i, t in enumerate(alone):
        for other in (together[i], out[i]):
            assert all(torch.equal(x, y) for x, y in zip(bytes_of(t), bytes_of(other))), i

    buf = torch.zeros(3000, device=DEV)
    for a, b in ((buf[:1000], buf[999:1999]), (buf[500:1500], buf[:501]), (buf[:1000], buf[8:108])):
        ts = [tw.AdamTensors.zero(x, state) for x in (a, b)]
        with pytest.raises(tw.TwellError):
            tw.adamw_step(ts, [torch.zeros_like(x) for x in (a, b)], 1, 1e-2)
    t, g = tw.AdamTensors.zero(buf[:1000], state), buf[999:1999]  # a gradient that the step writes into
    with pytest.raises(tw.TwellError):
        tw.adamw_step([t], [g], 1, 1e-2)
    with pytest.raises(tw.TwellError):
        tw.adamw_step([t], [torch.zeros(1000, device=DEV)], 1, 1e-2, grad_scale=buf[999:1000])
    assert (buf == 0).all()
