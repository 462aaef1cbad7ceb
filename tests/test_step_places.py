"""The optimizer's step on the host: what the binding hands over by default. No GPU is needed."""

import pytest

import activation_sparse_ffn_gate_amd as tw
from test_step_abi import calls  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("state", [torch.float32, torch.float8_e4m3fn])
def test_offset_by_default_is_the_step(calls, state):  # noqa: F811
    t, g = [tw.AdamTensors.zero(torch.zeros(300), state)], [torch.zeros(300)]
    for step, kw, want in ((1, {}, 1), (2, {}, 2), (1 << 40, {}, 1 << 40), (7, dict(offset=0), 0), (7, dict(offset=3), 3)):
        tw.adamw_step(t, g, step, 0.1, seed=5, **kw)
        assert calls[-1][1][-2:] == (5, want)
    with pytest.raises(ValueError, match="offset"):
        tw.adamw_step(t, g, 1, 0.1, offset=-1)
