"""Binding of the operators around the FFN (include/twell.h, "around the layer"):
dropout, residual addition with RMS norm, 4-bit products. Argument marshalling
only, as in _lib.py."""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

try:
    import torch
except ImportError:  # the package imports without torch; every call here takes its tensors
    torch = None

from ._lib import _Q4, _check, _workspace, lib

BF16, F32, E4M3 = 0, 1, 2
if torch is not None:
    _TYPES = {torch.bfloat16: BF16, torch.float32: F32, torch.float8_e4m3fn: E4M3}
    _FLOATS = (torch.bfloat16, torch.float32)
    _OUTS = (torch.bfloat16, torch.float8_e4m3fn)
    _XS = (torch.bfloat16, torch.float32, torch.float8_e4m3fn)


def _in(t, name, shape, dtypes, device):
    """Pointer of a contiguous tensor of one of `dtypes` on `device` (None for an empty one)."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _rows(x, name):
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, has {x.dim()}")
    return x.shape


def _bits64(v, name):
    if not 0 <= v < 1 << 64:
        raise ValueError(f"{name} must be in [0, 2^64), got {v}")
    return v


def _call(name, device, *args):
    """One entry point on the current stream of `device`."""
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    _check(st, name)


# ------------------------------------------------------------------ dropout and norm
def dropout(x, p: float, seed: int, offset: int = 0, residual=None, out=None, out_dtype=None):
    """twell_dropout: residual + dropout(x), the mask a function of (seed,
    offset, row, column) alone; the gradient's dropout is the same call on the
    gradient. out: a tensor to write (x or residual themselves are fine where
    the types are equal), else one of out_dtype (x's type by default)."""
    shape = _rows(x, "x")
    dev = x.device
    px = _in(x, "x", shape, _FLOATS, dev)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or (x.dtype if residual is None else residual.dtype), device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype says {out_dtype}")
    po = _in(out, "out", shape, _FLOATS, dev)
    pr = None if residual is None else _in(residual, "residual", shape, (out.dtype,), dev)
    _call("twell_dropout", dev, px, _TYPES[x.dtype], pr, shape[0], shape[1], p, _bits64(seed, "seed"),
          _bits64(offset, "offset"), po, _TYPES[out.dtype])
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
    shape = _rows(x, "x")
    dev = x.device
    M, d = shape
    px = _in(x, "x", shape, _FLOATS, dev)
    if h is None:
        if residual is None and p == 0 and h_dtype in (None, x.dtype):
            ph, h, th = None, x, x.dtype
        else:
            th = h_dtype or (x if residual is None else residual).dtype
            h = torch.empty(shape, dtype=th, device=dev)
            ph = _in(h, "h", shape, _FLOATS, dev)
    else:
        th = h.dtype
        if h_dtype is not None and th != h_dtype:
            raise TypeError(f"h is {th}, h_dtype says {h_dtype}")
        ph = _in(h, "h", shape, _FLOATS, dev)
    pr = None if residual is None else _in(residual, "residual", shape, (th,), dev)
    pw = _in(weight, "weight", (d,), _FLOATS, dev)
    out_dtype = out_dtype or torch.bfloat16
    n = torch.empty(shape, dtype=out_dtype, device=dev)
    pn = _in(n, "out", shape, _OUTS, dev)
    rstd = torch.empty(M, dtype=torch.float32, device=dev)
    scale = torch.empty(M, dtype=torch.float32, device=dev) if out_dtype is torch.float8_e4m3fn else None
    _call("twell_add_rmsnorm", dev, px, _TYPES[x.dtype], pr, pw, _TYPES[weight.dtype], M, d, eps, p,
          _bits64(seed, "seed"), _bits64(offset, "offset"), ph, _TYPES[th], pn, _TYPES[out_dtype],
          None if scale is None else scale.data_ptr() or None, rstd.data_ptr() or None)
    return Normed(n, h, rstd, scale)


def rmsnorm_workspace_bytes(M: int, d: int) -> int:
    return int(lib().twell_rmsnorm_workspace_bytes(M, d))


def add_rmsnorm_backward(dn, h, weight, rstd, dh=None, p: float = 0.0, seed: int = 0, offset: int = 0, dx_dtype=None,
                         workspace=None):
    """twell_add_rmsnorm_backward: (dres, dx, dweight) from the gradients of n
    and, where it has one, of h. dres has h's type, dx dx_dtype (h's by
    default); without dropout and of one type they are one tensor."""
    shape = _rows(dn, "dn")
    dev = dn.device
    M, d = shape
    pg = _in(dn, "dn", shape, _FLOATS, dev)
    ph = _in(h, "h", shape, _FLOATS, dev)
    pd = None if dh is None else _in(dh, "dh", shape, (h.dtype,), dev)
    pw = _in(weight, "weight", (d,), _FLOATS, dev)
    ps = _in(rstd, "rstd", (M,), (torch.float32,), dev)
    dres = torch.empty(shape, dtype=h.dtype, device=dev)
    dx, px = dres, None
    if p != 0 or dx_dtype not in (None, h.dtype):
        dx = torch.empty(shape, dtype=dx_dtype or h.dtype, device=dev)
        px = _in(dx, "dx", shape, _FLOATS, dev)
    dweight = torch.empty(d, dtype=torch.float32, device=dev)
    wp, wn = _workspace(workspace, dev).get(rmsnorm_workspace_bytes(M, d))
    _call("twell_add_rmsnorm_backward", dev, pg, _TYPES[dn.dtype], pd, ph, _TYPES[h.dtype], pw, _TYPES[weight.dtype],
          ps, M, d, p, _bits64(seed, "seed"), _bits64(offset, "offset"), dres.data_ptr() or None, px,
          _TYPES[dx.dtype], dweight.data_ptr() or None, wp, wn)
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
        if self.K != K or self.group != group:
            raise ValueError(f"{name} has K = {self.K}, group = {self.group}, expected {K}, {group}")
        if group <= 0:
            raise ValueError(f"{name} has group = {group}")
        per = (N, -(-K // group))
        return _Q4(
            _in(self.codes, f"{name}.codes", (N, -(-K // 2)), (torch.uint8,), device),
            _in(self.scales, f"{name}.scales", per, (torch.bfloat16,), device),
            None if self.zeros is None else _in(self.zeros, f"{name}.zeros", per, (torch.uint8,), device),
        )


def q4_quantize(W, group: int = 128) -> Q4:
    """twell_q4_quantize: round to nearest of a bf16 weight [N, K] of finite values."""
    N, K = _rows(W, "W")
    if group <= 0:
        raise ValueError(f"group must be positive, got {group}")
    pw = _in(W, "W", (N, K), (torch.bfloat16,), W.device)
    codes = torch.empty((N, -(-K // 2)), dtype=torch.uint8, device=W.device)
    scales = torch.empty((N, -(-K // group)), dtype=torch.bfloat16, device=W.device)
    _call("twell_q4_quantize", W.device, pw, N, K, group, codes.data_ptr() or None, scales.data_ptr() or None)
    return Q4(codes, scales, None, K, group)


def _q4_x(x, x_scale):
    M, K = _rows(x, "x")
    px = _in(x, "x", (M, K), _XS, x.device)
    if (x.dtype is torch.float8_e4m3fn) != (x_scale is not None):
        raise ValueError("x_scale goes with x in float8_e4m3fn, and only with it")
    ps = None if x_scale is None else _in(x_scale, "x_scale", (M,), (torch.float32,), x.device)
    return M, K, px, _TYPES[x.dtype], ps


def _q4_out(out, name, shape, dtype, device):
    if out is None:
        out = torch.empty(shape, dtype=dtype or torch.float32, device=device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"{name} is {out.dtype}, out_dtype says {dtype}")
    return out, _in(out, name, shape, _FLOATS, device)


def q4_workspace_bytes(x_dtype, M: int, N: int, K: int, gated: bool = False) -> int:
    return int(lib().twell_q4_workspace_bytes(_TYPES[x_dtype], M, N, K, gated))


def q4_matmul(x, W: Q4, x_scale=None, y=None, out_dtype=None, workspace=None):
    """twell_q4_matmul: y [M, N] = x W^T (float32 unless out_dtype or y says
    bfloat16). x bf16, float32, or e4m3 with x_scale [M] (add_rmsnorm's n, scale)."""
    M, K, px, xt, ps = _q4_x(x, x_scale)
    dev = x.device
    w = W._c("W", dev, W.N, K, W.group)
    y, py = _q4_out(y, "y", (M, W.N), out_dtype, dev)
    wp, wn = _workspace(workspace, dev).get(lib().twell_q4_workspace_bytes(xt, M, W.N, K, 0))
    _call("twell_q4_matmul", dev, px, xt, ps, ctypes.byref(w), M, W.N, K, W.group, py, _TYPES[y.dtype], wp, wn)
    return y


def q4_gateup(x, Wg: Q4, Wu: Q4, x_scale=None, h=None, out_dtype=None, workspace=None):
    """twell_q4_gateup: h [M, F] = z > 0 ? z u : 0, z = x Wg^T, u = x Wu^T."""
    M, K, px, xt, ps = _q4_x(x, x_scale)
    dev = x.device
    F, g = Wg.N, Wg.group
    wg, wu = Wg._c("Wg", dev, F, K, g), Wu._c("Wu", dev, F, K, g)
    h, ph = _q4_out(h, "h", (M, F), out_dtype, dev)
    wp, wn = _workspace(workspace, dev).get(lib().twell_q4_workspace_bytes(xt, M, F, K, 1))
    _call("twell_q4_gateup", dev, px, xt, ps, ctypes.byref(wg), ctypes.byref(wu), M, F, K, g, ph, _TYPES[h.dtype], wp,
          wn)
    return h


def ffn_q4_workspace_bytes(x_dtype, M: int, d: int, F: int) -> int:
    return int(lib().twell_ffn_q4_workspace_bytes(_TYPES[x_dtype], M, d, F))


def ffn_forward_q4(x, Wg: Q4, Wu: Q4, Wd: Q4, x_scale=None, y=None, workspace=None):
    """twell_ffn_forward_q4: the layer with 4-bit weights, y [M, d] float32.
    Wg and Wu are [F, d], Wd is [d, F] (down_proj.weight itself)."""
    M, d, px, xt, ps = _q4_x(x, x_scale)
    dev = x.device
    F, g = Wg.N, Wg.group
    wg, wu, wd = Wg._c("Wg", dev, F, d, g), Wu._c("Wu", dev, F, d, g), Wd._c("Wd", dev, d, F, g)
    y, py = _q4_out(y, "y", (M, d), torch.float32, dev)
    wp, wn = _workspace(workspace, dev).get(lib().twell_ffn_q4_workspace_bytes(xt, M, d, F))
    _call("twell_ffn_forward_q4", dev, px, xt, ps, ctypes.byref(wg), ctypes.byref(wu), ctypes.byref(wd), M, d, F, g, py,
          wp, wn)
    return y
