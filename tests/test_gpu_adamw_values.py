"""The optimizer's step: the draws of 8-bit states by default."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_adamw import DEV, E4M3, bytes_of, rand, state_of, values  # noqa: E402


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
