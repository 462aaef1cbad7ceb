"""4-bit products on the GPU: every kernel instance and its loop over K (the sizes
are those tests/test_q4_plan.py shows to reach them), exact cases, rows that hold
infinities and NaN.

Bounds, u = 2^-24. Per element as in tests/test_gpu_block.py: (K + 512) u of the sum
of magnitudes. Relative 2-norm over all elements, which shows an error that is
small in each: a rounding is 0.4 u of the partial sum (uniform over a unit in the
last place); 32 products are one partial sum, taken off a zero point as large as
the codes (8.8 rms beside 4.6 of q - z), in groups of up to 4 of them: 1.8 u of y
whatever K is; the K / g sums of a total add 0.4 u sqrt(K / 2 g) under 2.5 u. So
3 u for a product, 4.3 u for h = z u, 5.3 u for the FFN; six times that, 32 u =
1.9e-6, is the limit. (x in e4m3 by the matrix instruction of that format is off
by 1e-5.)"""

from __future__ import annotations

import numpy as np
import pytest

import _q4_plan as P
import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, U, q4_case, q4_x, rand  # noqa: E402

NAMES = {BF16: "bf16", F32: "f32", E4M3: "e4m3"}
NORM = 32 * U


def dev64(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(DEV)


def close64(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 1e-37)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def dot(x, w):
    """x w^T in fp64 on the device."""
    return torch.mm(x, w.t().contiguous())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K", P.WIDE + P.TILE)
def test_products(M, N, K, group, zeros):
    rng = np.random.default_rng(M + N + K + group)
    W, w = q4_case(rng, N, K, group, zeros)
    w = dev64(w)
    for xt in (BF16, F32, E4M3):
        print(f"[q4 product] {M}x{N}x{K} {P.instance(NAMES[xt], False, M, N, K, group)[0]} zeros {zeros}", flush=True)
        x, sx, xv = q4_x(rng, M, K, xt)
        xv = dev64(xv)
        big = torch.full((M * N + 128,), 7.0, dtype=F32, device=DEV)
        y = tw.q4_matmul(x, W, x_scale=sx, y=big[64:64 + M * N].view(M, N))
        want = dot(xv, w)
        close64(y, want, (K + 512) * U * dot(xv.abs(), w.abs()), "y")
        assert rel(y, want) < NORM
        assert (big[:64] == 7).all() and (big[-64:] == 7).all()
        assert torch.equal(y.to(BF16), tw.q4_matmul(x, W, x_scale=sx, out_dtype=BF16))  # the sums, rounded once


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,F,d", P.WIDE_GATED + P.TILE_GATED)
def test_gated_pairs(M, F, d, group, zeros):
    rng = np.random.default_rng(M + F + d + group)
    (Wg, wg), (Wu, wu) = q4_case(rng, F, d, group, zeros, True), q4_case(rng, F, d, group, zeros)
    wg, wu = dev64(wg), dev64(wu)
    for xt in (BF16, F32, E4M3):
        print(f"[q4 pair] {M}x{F}x{d} {P.instance(NAMES[xt], True, M, F, d, group)[0]} zeros {zeros}", flush=True)
        x, sx, xv = q4_x(rng, M, d, xt)
        xv = dev64(xv)
        z, u = dot(xv, wg), dot(xv, wu)
        zm, um = dot(xv.abs(), wg.abs()), dot(xv.abs(), wu.abs())
        want = torch.where(z > 0, z * u, 0.0)
        b = (d + 512) * U
        h = tw.q4_gateup(x, Wg, Wu, x_scale=sx)
        close64(h, want, b * (zm * u.abs() + um * z.abs()) + b * b * zm * um + 2 * U * want.abs(), "h")
        assert rel(h, want) < NORM
        assert torch.equal(h.to(BF16), tw.q4_gateup(x, Wg, Wu, x_scale=sx, out_dtype=BF16))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,d,F", P.FFN)
def test_ffn(M, d, F, group):
    rng = np.random.default_rng(M + F + d + group)
    zeros = bool(group & 64)
    (Wg, wg), (Wu, wu), (Wd, wd) = (q4_case(rng, F, d, group, zeros), q4_case(rng, F, d, group, zeros),
                                    q4_case(rng, d, F, group, zeros))
    wg, wu, wd = dev64(wg), dev64(wu), dev64(wd)
    for xt in (BF16, F32, E4M3):
        print(f"[q4 ffn] {M} rows d={d} F={F} {xt} down {P.ffn_instance(M, d, F, group)[0]}", flush=True)
        x, sx, xv = q4_x(rng, M, d, xt)
        xv = dev64(xv)
        z = dot(xv, wg)
        want = dot(torch.where(z > 0, z * dot(xv, wu), 0.0), wd)
        y = tw.ffn_forward_q4(x, Wg, Wu, Wd, x_scale=sx)
        assert rel(y, want) < NORM
        assert torch.equal(y, tw.ffn_forward_q4(x, Wg, Wu, Wd, x_scale=sx))


# ------------------------------------------------------------------ exact cases
def selection(rng, N, K, group, zero, scale=0.5):
    """A weight whose unit n is `scale` at column at[n] and zero elsewhere, with zero points of `zero`."""
    at = rng.integers(0, K, N)
    q = np.full((N, K), zero, dtype=np.uint8)
    q[np.arange(N), at] = zero + 1
    G = -(-K // group)
    z = None if zero == 8 else torch.full((N, G), zero, dtype=torch.uint8, device=DEV)
    s = torch.full((N, G), scale, dtype=BF16, device=DEV)
    return tw.Q4(torch.from_numpy(O.pack_codes(q)).to(DEV), s, z, K, group), torch.from_numpy(at).to(DEV)


@pytest.mark.parametrize("M,N,K,group", [(5, 300, 2100, 32), (40, 200, 1030, 64), (24, 8200, 1032, 32),
                                         (24, 8200, 1027, 64), (90, 7500, 1032, 128), (130, 7500, 1027, 32),
                                         (259, 8200, 520, 64)])
def test_selected_columns_come_through_exactly(M, N, K, group):
    """One term a unit: x times a power of two, with all 24 bits of a fp32 x. The
    other terms are zeros, whatever x has there, where z is 0, or goes into the codes."""
    rng = np.random.default_rng(M + N + K)
    for xt in (BF16, F32, E4M3):
        rows = 0 if P.plan(NAMES[xt], False, M, N, K, group).few else P.wide_rows(NAMES[xt], False, M, N)
        for zero in (0, 8) if xt == F32 or rows >= 64 else (0,):
            print(f"[q4 selection] {M}x{N}x{K} {xt} rows {rows} zero {zero}", flush=True)
            W, at = selection(rng, N, K, group, zero)
            x, sx, _ = q4_x(rng, M, K, xt)
            if xt == F32:  # bits of 24 places, values over many powers of two
                x = x * torch.from_numpy(2.0 ** rng.integers(-30, 30, (M, K))).to(DEV, F32)
            want = x.float()[:, at] * 0.5
            if sx is not None:
                want = want * sx[:, None]
            assert torch.equal(tw.q4_matmul(x, W, x_scale=sx), want)


@pytest.mark.parametrize("M,d,F,group", [(5, 300, 2100, 32), (7, 4201, 1100, 64), (40, 4100, 2100, 64),
                                         (90, 4100, 2101, 128)])
def test_hidden_values_keep_their_bits(M, d, F, group):
    """The FFN's y, where its down weight picks one hidden value a unit, is that of
    the gated pair in fp32, bit for bit."""
    rng = np.random.default_rng(M + d + F)
    (Wg, _), (Wu, _) = q4_case(rng, F, d, group, False), q4_case(rng, F, d, group, True)
    Wd, at = selection(rng, d, F, group, 8)
    for xt in (BF16, F32, E4M3):
        print(f"[q4 hidden] {M} rows d={d} F={F} {xt} {P.ffn_instance(M, d, F, group)[0]}", flush=True)
        x, sx, _ = q4_x(rng, M, d, xt)
        h = tw.q4_gateup(x, Wg, Wu, x_scale=sx)
        assert torch.equal(tw.ffn_forward_q4(x, Wg, Wu, Wd, x_scale=sx), h[:, at] * 0.5)


@pytest.mark.parametrize("M,N,K", [(4, 64, 256), (24, 8200, 1032), (90, 7500, 1027), (259, 8200, 520)])
def test_groups_of_one_large_weight(M, N, K):
    """Every group has one large weight, where x is zero, and zeros: y is zero. Where z
    goes into the codes that is exact; where it is a second product by the same x
    the two differ by the rounding of 32 terms x z: at most 32 u of their sum for each
    32 values of K."""
    rng = np.random.default_rng(M + K)
    group = 64
    for zero in (8, 13):
        q = np.full((N, K), zero, dtype=np.uint8)
        q[:, ::group] = 0
        z = None if zero == 8 else torch.full((N, -(-K // group)), zero, dtype=torch.uint8, device=DEV)
        s = torch.full((N, -(-K // group)), 0.3, dtype=BF16, device=DEV)
        W = tw.Q4(torch.from_numpy(O.pack_codes(q)).to(DEV), s, z, K, group)
        for xt in (BF16, F32, E4M3):
            x, sx, xv = q4_x(rng, M, K, xt)
            x[:, ::group] = 0
            xv[:, ::group] = 0
            few = P.plan(NAMES[xt], False, M, N, K, group).few
            pair = xt != F32 and (few or P.wide_rows(NAMES[xt], False, M, N) == 32)
            print(f"[q4 large weight] {M}x{N}x{K} {xt} zero {zero} pair {pair}", flush=True)
            y = tw.q4_matmul(x, W, x_scale=sx)
            if pair:
                assert (y.double().abs() <= dev64(np.abs(xv).sum(axis=1, keepdims=True)) * (32 * U * zero * 0.3011)).all()
            else:
                assert (y == 0).all()


# ------------------------------------------------------------------ infinities and NaN
@pytest.mark.parametrize("M,N,K", [(20, 50, 203), (24, 8200, 520), (24, 8200, 523), (80, 8200, 520), (80, 8200, 523),
                                   (259, 8200, 264)])
def test_rows_do_not_mix(M, N, K):
    """An infinity or NaN in one row of x, in its last, cut block among others, makes
    that row non-finite and leaves the others their bits."""
    rng = np.random.default_rng(M + K)
    W, _ = q4_case(rng, N, K, 64, True)
    V, _ = q4_case(rng, N, K, 64, False)
    for xt in (BF16, F32, E4M3):
        print(f"[q4 rows] {M}x{N}x{K} {P.instance(NAMES[xt], False, M, N, K, 64)[0]}", flush=True)
        x, sx, _ = q4_x(rng, M, K, xt)
        clean, pair = tw.q4_matmul(x, W, x_scale=sx), tw.q4_gateup(x, W, V, x_scale=sx)
        bad = [1, 3, M - 2]
        for r, k, v in zip(bad, (7, K - 1, K // 2), ("nan", "nan", "nan") if xt == E4M3 else ("nan", "inf", "-inf")):
            x[r, k] = float(v)
        rows = [r for r in range(M) if r not in bad]
        y, h = tw.q4_matmul(x, W, x_scale=sx), tw.q4_gateup(x, W, V, x_scale=sx)
        assert torch.equal(y[rows], clean[rows]) and torch.equal(h[rows], pair[rows])
        assert not torch.isfinite(y[bad]).any() and (h[1] == 0).all()


def test_x_at_an_odd_address():
    """bf16 rows of whole 16-byte pieces, one element past an aligned base."""
    rng = np.random.default_rng(12)
    for M, N, K in ((24, 8200, 520), (90, 7500, 1032), (9, 300, 264)):
        W, w = q4_case(rng, N, K, 64, True)
        x, _, xv = q4_x(rng, M, K, BF16)
        flat = torch.empty(M * K + 1, dtype=BF16, device=DEV)
        odd = flat[1:].view(M, K)
        odd.copy_(x)
        want, xv, w = dot(dev64(xv), dev64(w)), dev64(xv), dev64(w)
        for a in (x, odd):
            y = tw.q4_matmul(a, W)
            close64(y, want, (K + 512) * U * dot(xv.abs(), w.abs()), "y")
            assert rel(y, want) < NORM
