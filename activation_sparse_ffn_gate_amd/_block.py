"""Binding of the operators around the FFN (include/twell.h, "around the layer"):
dropout, residual addition with RMS norm, 4-bit products. Argument marshalling
only, as in _lib.py. The small calls of a decode step take less time on the GPU
than a few Python calls do, so each tensor is checked with one condition (_ptr)
and the reason is looked for only where it fails.

workspace: a Workspace of the caller's (calls that may run at the same time need
one each, and a graph's must stay as large as it was and live as long as the
graph), or None: scratch of this call alone."""

from __future__ import annotations

from ctypes import byref
from dataclasses import dataclass

from ._lib import _Q4, TwellError, lib

try:
    import torch
except ImportError:  # the package imports without torch; every call here takes its tensors
    torch = None
else:
    from torch import bfloat16, empty_like, float8_e4m3fn, float32, uint8

    _FLOATS = {bfloat16: 0, float32: 1}
    _OUTS = {bfloat16: 0, float8_e4m3fn: 2}
    _TYPES = {bfloat16: 0, float32: 1, float8_e4m3fn: 2}  # TWELL_BF16, TWELL_F32, TWELL_E4M3
    _F32, _BF16, _U8 = {float32: 1}, {bfloat16: 0}, {uint8: 3}


def _refuse(t, name, shape, dtypes, device):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t, name, shape, dtypes, device):
    """Address of a contiguous tensor of one of `dtypes` on `device` (0 for an empty one)."""
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != device.index or not t.is_contiguous():
        _refuse(t, name, shape, dtypes, device)
    return t.data_ptr()


def _rows(x, name, dtypes):
    """(device, shape, address) of a call's main operand, which has two dimensions."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, has {len(shape)}")
    if x.dtype not in dtypes or not x.is_contiguous():
        _refuse(x, name, shape, dtypes, x.device)
    return x.device, shape, x.data_ptr()


def _seeds(seed, offset):
    if not 0 <= seed < 1 << 64:
        raise ValueError(f"seed must be in [0, 2^64), got {seed}")
    if not 0 <= offset < 1 << 64:
        raise ValueError(f"offset must be in [0, 2^64), got {offset}")


def _call(fn, name, device, *args):
    """One entry point on the current stream of `device`."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        raise TwellError(st, name)


def _scratch(workspace, like, need):
    """(owner, address, bytes) of a call's scratch; the owner is held until the
    call is made. Without a workspace it is allocated here, on the current
    stream of the device of `like`, which the call runs on: no other stream or
    thread meets it, and in a capture it belongs to the graph's own memory."""
    if workspace is not None:
        if workspace.zeroed:
            raise ValueError("a control block must be a Workspace(zeroed=True) used for nothing else")
        if need:
            return workspace, *workspace.get(need)
    if not need:
        return None, None, 0
    buf = like.new_empty(need + 256, dtype=uint8)
    base = buf.data_ptr()
    return buf, base + -base % 256, need


# ------------------------------------------------------------------ dropout and norm
def dropout(x, p: float, seed: int, offset: int = 0, residual=None, out=None, out_dtype=None):
    """twell_dropout: residual + dropout(x), the mask a function of (seed,
    offset, row, column) alone; the gradient's dropout is the same call on the
    gradient. out: a tensor to write (x or residual themselves are fine where
    the types are equal), else one of out_dtype (residual's type by default, or x's)."""
    dev, shape, px = _rows(x, "x", _FLOATS)
    _seeds(seed, offset)
    if out is None:
        out_dtype = out_dtype or (x if residual is None else residual).dtype
        if out_dtype not in _FLOATS:
            raise TypeError(f"out must be torch.bfloat16 or torch.float32, got {out_dtype}")
        out = empty_like(x, dtype=out_dtype)
        po = out.data_ptr()
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype says {out_dtype}")
        po = _ptr(out, "out", shape, _FLOATS, dev)
    pr = None if residual is None else _ptr(residual, "residual", shape, (out.dtype,), dev)
    _call(lib().twell_dropout, "twell_dropout", dev, px, _FLOATS[x.dtype], pr, shape[0], shape[1], p, seed, offset, po,
          _FLOATS[out.dtype])
    return out


@dataclass
class Normed:
    """What add_rmsnorm gives: n [M, d] (bf16, or e4m3 whose row r stands for
    n[r] * scale[r]), h [M, d] the sum, rstd [M], scale [M] (None for bf16)."""

    n: "object"
    h: "object"
    rstd: "object"
    scale: "object" = None


def add_rmsnorm(x, weight, eps: float = 1e-6, residual=None, p: float = 0.0, seed: int = 0, offset: int = 0,
                out_dtype=None, h_dtype=None, h=None) -> Normed:
    """twell_add_rmsnorm: RMS norm of residual + dropout(x).

    out_dtype: torch.bfloat16 (the default), or torch.float8_e4m3fn with a scale a row. h:
    tensor for the sum (residual itself updates it in place), else one of
    residual's type, or without a residual of h_dtype (x's type by default).
    Without residual and dropout the sum is x, and h is x unless given."""
    dev, shape, px = _rows(x, "x", _FLOATS)
    _seeds(seed, offset)
    M, d = shape
    if h is None:
        if residual is None and p == 0 and h_dtype in (None, x.dtype):
            ph, h, th = None, x, x.dtype
        else:
            th = h_dtype or (x if residual is None else residual).dtype
            if th not in _FLOATS:
                raise TypeError(f"h must be torch.bfloat16 or torch.float32, got {th}")
            h = empty_like(x, dtype=th)
            ph = h.data_ptr()
    else:
        th = h.dtype
        if h_dtype is not None and th != h_dtype:
            raise TypeError(f"h is {th}, h_dtype says {h_dtype}")
        ph = _ptr(h, "h", shape, _FLOATS, dev)
    pr = None if residual is None else _ptr(residual, "residual", shape, (th,), dev)
    pw = _ptr(weight, "weight", (d,), _FLOATS, dev)
    out_dtype = out_dtype or bfloat16
    if out_dtype not in _OUTS:
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float8_e4m3fn, got {out_dtype}")
    n = empty_like(x, dtype=out_dtype)
    if out_dtype is bfloat16:
        rstd, scale, ps = x.new_empty(M, dtype=float32), None, None
    else:
        rstd, scale = x.new_empty((2, M), dtype=float32).unbind()
        ps = scale.data_ptr()
    _call(lib().twell_add_rmsnorm, "twell_add_rmsnorm", dev, px, _FLOATS[x.dtype], pr, pw, _FLOATS[weight.dtype], M, d,
          eps, p, seed, offset, ph, _FLOATS[th], n.data_ptr(), _OUTS[out_dtype], ps, rstd.data_ptr())
    return Normed(n, h, rstd, scale)


def rmsnorm_workspace_bytes(M: int, d: int) -> int:
    return int(lib().twell_rmsnorm_workspace_bytes(M, d))


def add_rmsnorm_backward(dn, h, weight, rstd, dh=None, p: float = 0.0, seed: int = 0, offset: int = 0, dx_dtype=None,
                         workspace=None):
    """twell_add_rmsnorm_backward: (dres, dx, dweight) from the gradients of n
    and, where it has one, of h. dres has h's type, dx dx_dtype (h's by
    default); without dropout and of one type they are one tensor."""
    dev, shape, pg = _rows(dn, "dn", _FLOATS)
    _seeds(seed, offset)
    M, d = shape
    th = h.dtype
    ph = _ptr(h, "h", shape, _FLOATS, dev)
    pd = None if dh is None else _ptr(dh, "dh", shape, (th,), dev)
    pw = _ptr(weight, "weight", (d,), _FLOATS, dev)
    ps = _ptr(rstd, "rstd", (M,), _F32, dev)
    dres = empty_like(h)
    dx, px = dres, None
    if p != 0 or dx_dtype not in (None, th):
        dx = empty_like(h, dtype=dx_dtype or th)
        px = _ptr(dx, "dx", shape, _FLOATS, dev)
    dweight = dn.new_empty(d, dtype=float32)
    L = lib()
    held, wp, wn = _scratch(workspace, dn, L.twell_rmsnorm_workspace_bytes(M, d))
    _call(L.twell_add_rmsnorm_backward, "twell_add_rmsnorm_backward", dev, pg, _FLOATS[dn.dtype], pd, ph, _FLOATS[th],
          pw, _FLOATS[weight.dtype], ps, M, d, p, seed, offset, dres.data_ptr(), px, _FLOATS[dx.dtype],
          dweight.data_ptr(), wp, wn)
    return dres, dx, dweight


# ------------------------------------------------------------------ 4-bit products
@dataclass
class Q4:
    """Device tensors of a weight [N, K] in 4 bits (see twell_q4 in include/twell.h)."""

    codes: "object"  # uint8 [N, ceil(K / 2)], k even in the low, k odd in the high 4 bits
    scales: "object"  # bfloat16 [N, ceil(K / group)]
    zeros: "object"  # uint8 [N, ceil(K / group)], or None: 8
    K: int
    group: int

    @property
    def N(self) -> int:
        return self.codes.shape[0]

    def _c(self, name, device, N, K, group):
        if self.K != K or self.group != group or group <= 0:
            raise ValueError(f"{name} has K = {self.K}, group = {self.group}, expected {K}, {group}")
        codes, scales, zeros = self.codes, self.scales, self.zeros
        rows, per, index = (N, (K + 1) // 2), (N, -(-K // group)), device.index
        if (codes.dtype is not uint8 or codes.shape != rows or codes.get_device() != index or not codes.is_contiguous()
                or scales.dtype is not bfloat16 or scales.shape != per or scales.get_device() != index
                or not scales.is_contiguous()):
            _ptr(codes, f"{name}.codes", rows, _U8, device)
            _refuse(scales, f"{name}.scales", per, _BF16, device)
        return _Q4(codes.data_ptr(), scales.data_ptr(),
                   None if zeros is None else _ptr(zeros, "zeros", per, _U8, device))


def q4_quantize(W, group: int = 128) -> Q4:
    """twell_q4_quantize: round to nearest of a bf16 weight [N, K] of finite values."""
    if group <= 0:
        raise ValueError(f"group must be positive, got {group}")
    dev, (N, K), pw = _rows(W, "W", _BF16)
    codes = W.new_empty((N, (K + 1) // 2), dtype=uint8)
    scales = W.new_empty((N, -(-K // group)))
    _call(lib().twell_q4_quantize, "twell_q4_quantize", dev, pw, N, K, group, codes.data_ptr(), scales.data_ptr())
    return Q4(codes, scales, None, K, group)


def _q4_scale(x, x_scale, M, dev):
    if x_scale is None:
        if x.dtype is float8_e4m3fn:
            raise ValueError("x in float8_e4m3fn needs x_scale")
        return None
    if x.dtype is not float8_e4m3fn:
        raise ValueError("x_scale goes with x in float8_e4m3fn only")
    return _ptr(x_scale, "x_scale", (M,), _F32, dev)


def _q4_out(out, name, x, shape, dtype, dev):
    if out is None:
        dtype = dtype or float32
        if dtype not in _FLOATS:
            raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        out = x.new_empty(shape, dtype=dtype)
        return out, out.data_ptr()
    if dtype is not None and out.dtype != dtype:
        raise TypeError(f"{name} is {out.dtype}, out_dtype says {dtype}")
    return out, _ptr(out, name, shape, _FLOATS, dev)


def q4_workspace_bytes(x_dtype, M: int, N: int, K: int, gated: bool = False) -> int:
    return int(lib().twell_q4_workspace_bytes(_TYPES[x_dtype], M, N, K, gated))


def q4_matmul(x, W: Q4, x_scale=None, y=None, out_dtype=None, workspace=None):
    """twell_q4_matmul: y [M, N] = x W^T (float32 unless out_dtype or y says
    bfloat16). x bf16, float32, or e4m3 with x_scale [M] (add_rmsnorm's n, scale)."""
    dev, (M, K), px = _rows(x, "x", _TYPES)
    xt, ps = _TYPES[x.dtype], _q4_scale(x, x_scale, M, dev)
    N, g = W.N, W.group
    w = W._c("W", dev, N, K, g)
    y, py = _q4_out(y, "y", x, (M, N), out_dtype, dev)
    L = lib()
    held, wp, wn = _scratch(workspace, x, L.twell_q4_workspace_bytes(xt, M, N, K, 0))
    _call(L.twell_q4_matmul, "twell_q4_matmul", dev, px, xt, ps, byref(w), M, N, K, g, py, _FLOATS[y.dtype], wp, wn)
    return y


def q4_gateup(x, Wg: Q4, Wu: Q4, x_scale=None, h=None, out_dtype=None, workspace=None):
    """twell_q4_gateup: h [M, F] = z > 0 ? z u : 0, z = x Wg^T, u = x Wu^T."""
    dev, (M, K), px = _rows(x, "x", _TYPES)
    xt, ps = _TYPES[x.dtype], _q4_scale(x, x_scale, M, dev)
    F, g = Wg.N, Wg.group
    wg, wu = Wg._c("Wg", dev, F, K, g), Wu._c("Wu", dev, F, K, g)
    h, ph = _q4_out(h, "h", x, (M, F), out_dtype, dev)
    L = lib()
    held, wp, wn = _scratch(workspace, x, L.twell_q4_workspace_bytes(xt, M, F, K, 1))
    _call(L.twell_q4_gateup, "twell_q4_gateup", dev, px, xt, ps, byref(wg), byref(wu), M, F, K, g, ph, _FLOATS[h.dtype],
          wp, wn)
    return h


def ffn_q4_workspace_bytes(x_dtype, M: int, d: int, F: int) -> int:
    return int(lib().twell_ffn_q4_workspace_bytes(_TYPES[x_dtype], M, d, F))


def ffn_forward_q4(x, Wg: Q4, Wu: Q4, Wd: Q4, x_scale=None, y=None, workspace=None):
    """twell_ffn_forward_q4: the layer with 4-bit weights, y [M, d] float32.
    Wg and Wu are [F, d], Wd is [d, F] (down_proj.weight itself)."""
    dev, (M, d), px = _rows(x, "x", _TYPES)
    xt, ps = _TYPES[x.dtype], _q4_scale(x, x_scale, M, dev)
    F, g = Wg.N, Wg.group
    wg, wu, wd = Wg._c("Wg", dev, F, d, g), Wu._c("Wu", dev, F, d, g), Wd._c("Wd", dev, d, F, g)
    y, py = _q4_out(y, "y", x, (M, d), float32, dev)
    L = lib()
    held, wp, wn = _scratch(workspace, x, L.twell_ffn_q4_workspace_bytes(xt, M, d, F))
    _call(L.twell_ffn_forward_q4, "twell_ffn_forward_q4", dev, px, xt, ps, byref(wg), byref(wu), byref(wd), M, d, F, g,
          py, wp, wn)
    return y
