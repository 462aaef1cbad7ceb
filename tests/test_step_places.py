"""The optimizer's step and the adapters on the host: what the binding hands over by default, and memory that is
written and belongs to something else too. No GPU is needed."""

import pytest

import activation_sparse_ffn_gate_amd as tw
from activation_sparse_ffn_gate_amd._lib import _AdamwTensor
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


N, E_ARG = 1000, -1
BASE = 1 << 40  # never dereferenced: what is listed here is refused


def _step(tensors, e4m3, grad_scale=None):
    """Status of a step of tensors given as {field: address}; places not given lie 64 KB apart, each alone."""
    made = []
    for i, fields in enumerate(tensors):
        at = {k: BASE + (16 * i + j) * 65536 for j, (k, _) in enumerate(_AdamwTensor._fields_[:12])}
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            at[k + "_out"] = at[k]  # in place
        at |= fields
        if not e4m3:
            at |= dict.fromkeys(("m_scale", "v_scale", "m_scale_out", "v_scale_out"))
        made.append(_AdamwTensor(**at, n=N, weight_decay=0.0, g_type=1))
    return tw.lib().twell_adamw((_AdamwTensor * len(made))(*made), len(made), 2 if e4m3 else 1, 1, 1e-3, 0.9, 0.99, 1e-8,
                                grad_scale, 1, 2, None)


def _at(i, k):
    return BASE + (16 * i + [f for f, _ in _AdamwTensor._fields_].index(k)) * 65536


@pytest.mark.parametrize("e4m3", [False, True])
def test_adamw_refuses_memory_of_two_tensors(e4m3):
    """Wholly and in part, at either end, within one tensor and between the first and the last of many. (What is allowed
    needs memory: the tests on the GPU.)"""
    state = N if e4m3 else 4 * N
    size = dict(p=4 * N, m=state, v=state, copy=2 * N, g=4 * N) | (dict(m_scale=16, v_scale=16) if e4m3 else {})
    written = [k for k in size if k != "g"]
    for a in written:
        for b in size:
            for other in (0, 1, 40):  # the tensor that has b
                if other == 0 and a == b:
                    continue
                place = "copy" if a == "copy" else a + "_out"
                ends = [_at(other, b) - size[a] + 4, _at(other, b) + size[b] - 4, _at(other, b) + 4]
                if other:
                    ends.append(_at(other, b))
                for address in ends:
                    tensors = [{place: address}] + [{}] * other
                    assert _step(tensors, e4m3) == E_ARG, (a, b, other, address - _at(other, b))
    # an old value where another tensor writes, or in part where its own does
    for k in written[:3]:
        for address in (_at(1, k), _at(1, k) + 8, _at(0, k) + 8, _at(0, k) - 8):
            assert _step([{k: address, k + "_out": _at(0, k)}, {}], e4m3) == E_ARG, (k, address)
    for k in written:
        assert _step([{}, {}], e4m3, _at(1, k) + size[k] - 4) == E_ARG, k


@pytest.mark.parametrize("x_type,y_type", [(0, 1), (1, 0), (2, 1)])
def test_lora_refuses_y_in_other_operands(x_type, y_type):
    """In part, at either end, and inside."""
    M, N, K, R, n = 5, 200, 72, 7, 3
    x_size, y_size = {0: 2, 1: 4, 2: 1}, {0: 2, 1: 4}
    sizes = dict(x=M * K * x_size[x_type], x_scale=4 * M, index=4 * M, A=2 * n * R * K, B=2 * n * N * R, scaling=4 * n,
                 base=M * N * y_size[y_type])
    at = {k: BASE + i * 65536 for i, k in enumerate(sizes)}

    def call(y):
        a = at | (dict(x_scale=None) if x_type != 2 else {})
        return tw.lib().twell_lora(a["x"], x_type, a["x_scale"], a["index"], a["A"], a["B"], a["scaling"], n, M, N, K, R, a["base"], y,
                                   y_type, None)

    for k, size in sizes.items():
        if k == "x_scale" and x_type != 2:
            continue
        for y in [at[k] - sizes["base"] + 1, at[k] + size - 1, at[k] + 4] + ([at[k]] if k != "base" else []):
            assert call(y) == E_ARG, (k, y - at[k])
