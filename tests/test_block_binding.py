"""Binding of the operators around the FFN: what it hands to the C entry points.
No GPU is needed: the calls are recorded and not made."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from activation_sparse_ffn_gate_amd import _block, _lib  # noqa: E402

CPU = torch.device("cpu")


@pytest.fixture
def calls(monkeypatch):
    """Entry points that record their arguments in a list, on host tensors.
    calls.inside: run once while the first call is being made."""

    class Calls(list):
        inside = None

    seen = Calls()

    def call(fn, name, device, *args):
        seen.append((name, args))
        if seen.inside is not None:
            inside, seen.inside = seen.inside, None
            inside()

    monkeypatch.setattr(_block, "_call", call)
    monkeypatch.setattr(_block, "_rows", lambda x, name, dtypes: (x.device, x.shape, x.data_ptr()))
    monkeypatch.setattr(_block, "_ptr", lambda t, name, shape, dtypes, device: t.data_ptr())
    monkeypatch.setattr(_block.Q4, "_c", lambda self, *a: _block._Q4(1, 1, 0))
    return seen


def _q4(N, K):
    return tw.Q4(torch.empty(N, K // 2, dtype=torch.uint8), None, None, K, 32)


def _ffn(M, d=64, F=96, **kw):
    return lambda: tw.ffn_forward_q4(torch.zeros(M, d, dtype=torch.bfloat16), _q4(F, d), _q4(F, d), _q4(d, F), **kw)


def _product(M, **kw):  # K long enough to be split: partial sums
    return lambda: tw.q4_matmul(torch.zeros(M, 1 << 14, dtype=torch.bfloat16), _q4(32, 1 << 14), **kw)


def _pair(M, **kw):
    w = _q4(64, 1 << 14)
    return lambda: tw.q4_gateup(torch.zeros(M, 1 << 14, dtype=torch.bfloat16), w, w, **kw)


def _norm_backward(M, d=64, **kw):
    x = torch.zeros(M, d)
    return lambda: tw.add_rmsnorm_backward(x, x, torch.ones(d), torch.ones(M), **kw)


def _span(call):
    address, size = call[1][-2:]
    address = getattr(address, "value", address)
    return address, address + size


@pytest.mark.parametrize("make", [_ffn, _product, _pair, _norm_backward])
@pytest.mark.parametrize("sizes", [(4, 4), (4, 300), (300, 4)])
def test_calls_under_way_together_have_their_own_scratch(calls, make, sizes):
    """Another stream's or thread's call, made while one is under way, writes
    elsewhere, and does not take the first one's memory away by needing more."""
    calls.inside = make(sizes[1])
    make(sizes[0])()
    (a0, a1), (b0, b1) = _span(calls[0]), _span(calls[1])
    assert a1 > a0 and b1 > b0 and a0 % 256 == 0 and b0 % 256 == 0
    assert a1 <= b0 or b1 <= a0


def test_scratch_is_not_the_packing_that_a_forward_left(calls):
    """tw.packed_view reads what twell_ffn_forward left in the default workspace."""
    left = _lib._workspace(None, CPU)
    left.get(1 << 22)
    left.buf.fill_(7)
    held = left.buf
    _ffn(300)()
    lo, hi = _span(calls[0])
    assert left.buf is held and (hi <= held.data_ptr() or held.data_ptr() + held.numel() <= lo)


@pytest.mark.parametrize("make", [_ffn, _product, _pair, _norm_backward])
def test_a_workspace_of_the_callers_is_used(calls, make):
    ws = tw.Workspace(CPU)
    make(4, workspace=ws)()
    lo, hi = _span(calls[0])
    assert ws.buf.data_ptr() <= lo and hi <= ws.buf.data_ptr() + ws.buf.numel()
    with pytest.raises(ValueError, match="control block"):
        make(4, workspace=tw.Workspace(CPU, zeroed=True))()
