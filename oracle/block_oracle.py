"""Plain fp64 CPU oracle of the operators around the FFN: dropout, residual
addition with RMS or layer norm and its gradients, 4-bit weights and their products,
low-rank adapters, the optimizer's step.

TEST INFRASTRUCTURE ONLY (see the package docstring). Inputs are numpy arrays
of values (bf16 decoded with decode_bf16), results fp64 and not rounded to any
output type, except where a function says so.
"""

from __future__ import annotations

import math

import numpy as np

_M32 = (1 << 32) - 1


def philox4x32(counter, key, rounds: int = 10):
    """Philox4x32 of one counter (4 words) and key (2 words) in Python integers
    (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & _M32, (a >> 32) ^ c[3] ^ k[1], a & _M32]
        k = [(k[0] + 0x9E3779B9) & _M32, (k[1] + 0xBB67AE85) & _M32]
    return tuple(c)


def keep_threshold(p: float) -> int:
    """Kept: 16 bits >= floor(65536 p + 1/2)."""
    return int(math.floor(65536 * p + 0.5))


def keep_mask(M: int, d: int, p: float, seed: int, offset: int, rows=None) -> np.ndarray:
    """bool [M, d] (or the given rows): element (r, c) has 16-bit half c % 2
    (0 the low one) of word (c % 8) / 2 of the generator at counter
    (c / 8, r, offset low, offset high), key (seed low, seed high)."""
    t = keep_threshold(p)
    rows = range(M) if rows is None else rows
    out = np.empty((len(rows), d), dtype=bool)
    for i, r in enumerate(rows):
        for b in range(-(-d // 8)):
            w = philox4x32((b, r, offset & _M32, offset >> 32), (seed & _M32, seed >> 32))
            for j in range(min(8, d - 8 * b)):
                out[i, 8 * b + j] = ((w[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= t
    return out


def dropout(x, p, seed, offset, residual=None, keep=None):
    """residual + kept x / (probability of being kept, as realised)."""
    keep = keep_mask(*x.shape, p, seed, offset) if keep is None else keep
    y = np.where(keep, x * (65536.0 / (65536 - keep_threshold(p))), 0.0)
    return y if residual is None else residual + y


def rmsnorm(s, weight, eps):
    """(s rstd weight, rstd) with rstd = 1 / sqrt(mean(s^2) + eps) a row."""
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    return s * rstd[:, None] * weight, rstd


def rmsnorm_backward(dout, h, weight, rstd):
    """(gradient of h, gradient of weight) of sum(dout * rmsnorm(h))."""
    g = dout * weight
    c = (g * h).sum(axis=1) * rstd**3 / h.shape[1]
    return rstd[:, None] * g - c[:, None] * h, (dout * h * rstd[:, None]).sum(axis=0)


def layernorm(s, weight, bias, eps):
    """((s - mean) rstd weight + bias, mean, rstd) with rstd = 1 / sqrt(mean((s - mean)^2) + eps) a row."""
    mean = s.mean(axis=1)
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    return c * rstd[:, None] * weight + (0.0 if bias is None else bias), mean, rstd


def layernorm_backward(dout, h, weight, mean, rstd):
    """(gradient of h, of weight, of bias) of sum(dout * layernorm(h))."""
    g = dout * weight
    xh = (h - mean[:, None]) * rstd[:, None]
    ds = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    return ds, (dout * xh).sum(axis=0), dout.sum(axis=0)


def lora(x, index, A, B, scaling, base):
    """base + scaling[a] (x A[a]^T) B[a]^T, a = index[row]; base where that names no adapter."""
    y = base.copy()
    for m, a in enumerate(index):
        if 0 <= a < len(A):
            y[m] += scaling[a] * (B[a] @ (A[a] @ x[m]))
    return y


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after step `step` (from 1)."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1**step)) / (np.sqrt(v / (1 - beta2**step)) + eps)
    return p - lr * (weight_decay * p + hat), m, v


def state_bits(n, number, seed, offset):
    """16 bits for each element of tensor `number`: dropout's, with the tensor as the row."""
    out = np.empty(-(-n // 8) * 8, dtype=np.int64)
    for b in range(-(-n // 8)):
        w = philox4x32((b, number, offset & _M32, offset >> 32), (seed & _M32, seed >> 32))
        for j in range(8):
            out[8 * b + j] = (w[j // 2] >> (16 * (j % 2))) & 0xFFFF
    return out[:n]


def block_scales(v, block=256):
    """max(largest |value|, 2^-100) / 448 of each block of consecutive elements."""
    return np.array([max(np.abs(v[i:i + block]).max(), 2.0**-100) / 448 for i in range(0, len(v), block)])


def to_neighbour(x, bits, least=0.0):
    """x (|x| <= 448) to its e4m3 neighbour above (in magnitude) where (bits + 1/2) / 256 is at least
    one minus its place between the two, else below; what is not zero is at least `least`."""
    grid = e4m3_values()[:127]  # 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    at = np.searchsorted(grid, a, side="right") - 1
    above = grid[np.minimum(at + 1, 126)]
    gap = np.where(above > grid[at], above - grid[at], 1.0)
    q = np.where((a - grid[at]) / gap >= 1 - (bits + 0.5) / 256, above, grid[at])
    return np.sign(x) * np.where(a > 0, np.maximum(q, least), 0.0)


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP e4m3: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 0 is subnormal, S.1111.111 is NaN, there is no infinity."""
    v = np.empty(256)
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        mag = m * 2.0**-9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[i] = (-mag if i & 128 else mag) if i & 127 != 127 else np.nan
    return v


def q4_quantize(W, group):
    """(codes 0..15 [N, K], scales [N, G] as bf16 values): scale = max|W| / 7 of
    the group rounded to bf16 (nearest even), code = round(W / scale) + 8 clamped;
    division and rounding in fp32, as the kernel states them."""
    N, K = W.shape
    G = -(-K // group)
    codes, scales = np.full((N, K), 8, dtype=np.uint8), np.zeros((N, G))
    for g in range(G):
        w = W[:, g * group:(g + 1) * group].astype(np.float32)
        s = _round_bf16(np.abs(w).max(axis=1) / np.float32(7))
        scales[:, g] = s
        live = s > 0
        q = np.rint(w[live] / s[live, None].astype(np.float32)) + 8
        codes[live, g * group:(g + 1) * group] = np.clip(q, 0, 15)
    return codes, scales


def _round_bf16(a):
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def pack_codes(q):
    """codes [N, K] -> bytes [N, ceil(K / 2)]: k even in the low, k odd in the high 4 bits."""
    N, K = q.shape
    full = np.zeros((N, K + K % 2), dtype=np.uint8)
    full[:, :K] = q
    return full[:, 0::2] | (full[:, 1::2] << 4)


def q4_dequantize(codes, scales, zeros, group):
    """scales (q - zeros) with codes [N, K] one a byte; zeros None: 8."""
    g = np.arange(codes.shape[1]) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[:, g]
    return scales[:, g] * (codes.astype(np.float64) - z)


def gated_hidden(x, Wg, Wu):
    """z > 0 ? z u : 0, z = x Wg^T, u = x Wu^T (fp64 weights [F, d])."""
    z, u = x @ Wg.T, x @ Wu.T
    return np.where(z > 0, z * u, 0.0)
