"""Binding of the optimizer's step (include/twell.h, "the optimizer's step"): the
norm of all gradients with the factor that clips it, and AdamW over many tensors in
one call. Argument marshalling only, as in _block.py. The step's number, lr and offset are launch
arguments: a captured graph repeats the step that it was captured with."""

from __future__ import annotations

import struct
from dataclasses import dataclass

from ._block import _BF16, _F32, _FLOATS, _call, _ptr, _refuse, _scratch, _seeds
from ._lib import lib

try:
    import torch
except ImportError:  # the package imports without torch; every call here takes its tensors
    torch = None
else:
    from torch import bfloat16, float8_e4m3fn, float32

    _STATES = {float32: 1, float8_e4m3fn: 2}  # TWELL_F32, TWELL_E4M3

# Elements of the arrays that the C entries read (_lib._Grad, _lib._AdamwTensor)
_GRAD, _TENSOR = struct.Struct("Qqi4x").pack, struct.Struct("12Qqdi4x").pack

STATE_BLOCK = 256  # elements of an 8-bit state that share a scale


@dataclass(slots=True)
class AdamTensors:
    """Device tensors of one parameter, all of its shape but the scales: p its fp32
    values, m and v the moments in float32, or in float8_e4m3fn with m_scale and v_scale
    float32 [ceil(numel / 256)] (then m * scale, and v's root: see twell_adamw_tensor in include/twell.h),
    copy a bfloat16 tensor that receives the new p, or None."""

    p: "object"
    m: "object"
    v: "object"
    m_scale: "object" = None
    v_scale: "object" = None
    copy: "object" = None

    @classmethod
    def zero(cls, p, state_dtype=None, copy=None):
        """The state before the first step."""
        m, v = (torch.zeros_like(p, dtype=state_dtype or float32) for _ in range(2))
        if m.dtype is not float8_e4m3fn:
            return cls(p, m, v, copy=copy)
        scales = torch.zeros((2, -(-p.numel() // STATE_BLOCK)), dtype=float32, device=p.device)
        return cls(p, m, v, *scales.unbind(), copy=copy)

    def _refuse(self, name, g, state, dev):
        """Why _addresses took these tensors for unfit."""
        shape, scales = g.shape, (-(-g.numel() // STATE_BLOCK),)
        _ptr(self.p, f"{name}.p", shape, _F32, dev)
        _ptr(self.m, f"{name}.m", shape, (state,), dev)
        _ptr(self.v, f"{name}.v", shape, (state,), dev)
        for k, t in (("m_scale", self.m_scale), ("v_scale", self.v_scale)):
            if (t is None) != (state is float32):
                raise ValueError(f"{name}.{k}: scales go with states in float8_e4m3fn, and only with them")
            if t is not None:
                _ptr(t, f"{name}.{k}", scales, _F32, dev)
        _refuse(self.p, name, shape, _F32, dev)


def _addresses(t, g, n, state, index):
    """p, m, v, m_scale, v_scale of an AdamTensors fit for gradient g (one condition: these are many
    tensors in a call), or None."""
    p, m, v, ms, vs = t.p, t.m, t.v, t.m_scale, t.v_scale
    if (p.dtype is not float32 or m.dtype is not state or v.dtype is not state or not p.is_same_size(g)
            or not m.is_same_size(g) or not v.is_same_size(g) or p.get_device() != index or m.get_device() != index
            or v.get_device() != index or not p.is_contiguous() or not m.is_contiguous() or not v.is_contiguous()):
        return None
    if state is float32:
        return (p.data_ptr(), m.data_ptr(), v.data_ptr(), 0, 0) if ms is None and vs is None else None
    blocks = (-(-n // STATE_BLOCK),)
    for s in (ms, vs):
        if (s is None or s.dtype is not float32 or s.shape != blocks or s.get_device() != index
                or not s.is_contiguous()):
            return None
    return p.data_ptr(), m.data_ptr(), v.data_ptr(), ms.data_ptr(), vs.data_ptr()


def _device(tensors, name):
    if not tensors:
        raise ValueError(f"{name} is empty")
    if not tensors[0].is_cuda:
        raise ValueError(f"{name}[0] must be a device tensor")
    return tensors[0].device


def _grads(grads, dev):
    """(list for the C entry, count)"""
    rows = [_GRAD(_ptr(g, "a gradient", g.shape, _FLOATS, dev), g.numel(), _FLOATS[g.dtype]) for g in grads]
    return b"".join(rows), len(grads)


def grad_norm_workspace_bytes(grads) -> int:
    return int(lib().twell_grad_norm_workspace_bytes(*_grads(grads, _device(grads, "grads"))))


def grad_norm(grads, max_norm: float = float("inf"), out=None, workspace=None):
    """twell_grad_norm: float32 [2], the 2-norm of all gradients (bf16 or float32) together and
    min(1, max_norm / norm); out[1:] is adamw_step's grad_scale, with no wait for the device between."""
    grads = list(grads)
    dev = _device(grads, "grads")
    listed, count = _grads(grads, dev)
    if out is None:
        out = torch.empty(2, dtype=float32, device=dev)
        po = out.data_ptr()
    else:
        po = _ptr(out, "out", (2,), _F32, dev)
    L = lib()
    held, wp, wn = _scratch(workspace, out, L.twell_grad_norm_workspace_bytes(listed, count))
    _call(L.twell_grad_norm, "twell_grad_norm", dev, listed, count, max_norm, po, wp, wn)
    return out


def adamw_step(tensors, grads, step: int, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0,
               grad_scale=None, seed: int = 0, offset: int | None = None, out=None):
    """twell_adamw: step `step` (from 1) of a list of AdamTensors, in place, with one gradient each (bf16 or
    float32, of p's shape). weight_decay: a number, or one a tensor. grad_scale: float32 [1] on the
    device that multiplies the gradients (grad_norm's out[1:]; 0, NaN or infinity: the step is
    skipped, and nothing is written, to out neither). seed, offset: of the rounding of 8-bit states, whose draws have to be others each step (with
    the same ones, second moments stop falling); offset is the step's number unless given. out: a
    list of AdamTensors that receive the new values instead (and their copies). Memory that two
    tensors write, or that one writes and another reads, is refused, in part too."""
    grads = list(grads)
    dev = _device(grads, "grads")
    if offset is None:
        offset = max(step, 0)
    _seeds(seed, offset)
    count, index = len(tensors), dev.index
    if len(grads) != count or (out is not None and len(out) != count):
        raise ValueError(f"{count} tensors, {len(grads)} gradients" + ("" if out is None else f", {len(out)} outputs"))
    decays = [weight_decay] * count if isinstance(weight_decay, (int, float)) else list(weight_decay)
    if len(decays) != count:
        raise ValueError(f"{count} tensors, {len(decays)} weight decays")
    state = tensors[0].m.dtype
    if state not in _STATES:
        raise TypeError(f"states must be torch.float32 or torch.float8_e4m3fn, got {state}")
    listed, written, read, kept = [], [], [], 3 if state is float32 else 5
    for t, to, g, decay in zip(tensors, out or tensors, grads, decays):
        n, i = g.numel(), len(listed)
        g_type = _FLOATS.get(g.dtype)
        if g_type is None or g.get_device() != index or not g.is_contiguous():
            _ptr(g, "a gradient", g.shape, _FLOATS, dev)
        pg = g.data_ptr()
        old = _addresses(t, g, n, state, index)
        if old is None:
            t._refuse(f"tensors[{i}]", g, state, dev)
        new = old
        if to is not t:
            new = _addresses(to, g, n, state, index)
            if new is None:
                to._refuse(f"out[{i}]", g, state, dev)
        copy = 0
        if (c := to.copy) is not None:
            if c.dtype is not bfloat16 or not c.is_same_size(g) or c.get_device() != index or not c.is_contiguous():
                _ptr(c, "copy", g.shape, _BF16, dev)
            copy = c.data_ptr()
        if n:
            written += new[:kept]
            if copy:
                written.append(copy)
            read.append(pg)
            if to is not t:
                read += [a for a in old[:kept] if a not in new]
        listed.append(_TENSOR(old[0], pg, *old[1:], *new, copy, n, decay, g_type))
    places = set(written)
    if len(places) != len(written):
        raise ValueError("a tensor is listed twice")
    if not places.isdisjoint(read):
        raise ValueError("a tensor that receives new values is a gradient or another one's old value")
    ps = None if grad_scale is None else _ptr(grad_scale, "grad_scale", (1,), _F32, dev)
    _call(lib().twell_adamw, "twell_adamw", dev, b"".join(listed), count, _STATES[state], step, lr, *betas, eps, ps, seed,
          offset)
