"""Operators around the FFN on the GPU, through the binding, against the fp64
oracle at the sizes, types and values where they can go wrong.

Error bounds, per element and derived from the arithmetic, u = 2^-24:
* bf16 output: 2^-8 of the value (half a unit in the last place of 8 significant
  bits) on top of the fp32 result's error; e4m3: 2^-4 of it, at least 2^-10 (half
  the subnormal step).
* sums: a chain of n fp32 additions of terms a_i is off by at most n u sum|a_i|.
  The norm's longest chain is 64 terms a thread and 8 levels across threads;
  with the operations around it 2^-17 of the sum of magnitudes is over 128 u.
* dweight: at most M / 512 rows a workgroup, 4 waves, 16 + 5 additions of the
  second step: under 256 u = 2^-16 for the sizes here.
* 4-bit products: 32 products a matrix instruction (taken as 32 additions), K / 32
  of them, the groups' sums and the waves': under (K + 512) u.
"""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402

DEV = torch.device("cuda", 0)
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0**-24
SUM = 2.0**-17
SEED, OFFSET = 0x123456789ABCDEF0, (7 << 32) + 3


def host(t):
    return t.double().cpu().numpy()


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype).to(DEV)


def half_step(dtype, v):
    """Largest rounding of v to dtype."""
    if dtype == F32:
        return U * np.abs(v)
    if dtype == BF16:
        return 2.0**-8 * np.abs(v)
    return np.maximum(2.0**-4 * np.abs(v), 2.0**-10)


def close(got, want, bound, what):
    got = host(got) if isinstance(got, torch.Tensor) else got
    err = np.abs(got - want)
    bad = ~(err <= bound + 1e-37)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}")


# rows and widths: one, odd, cut blocks, both sides of every choice of shape (512, 2048, 4096,
# 8192, 16384 columns; 2048 rows), the layers' widths
SIZES = [(1, 1), (3, 7), (5, 8), (4, 9), (1, 2048), (7, 511), (6, 513), (2049, 40), (2050, 1000), (2051, 2048),
         (9, 2049), (5, 2560), (3, 4097), (4, 8192), (2, 8193), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("xt,yt,p,res", [(F32, BF16, 0.1, False), (BF16, F32, 0.5, True), (BF16, BF16, 0.9, True),
                                         (F32, F32, 0.0, False)])
def test_dropout(M, d, xt, yt, p, res):
    print(f"[dropout] {M}x{d} {xt} {yt} p={p}", flush=True)
    rng = np.random.default_rng(M * 7 + d)
    x = rand(rng, (M, d), xt)
    r = rand(rng, (M, d), yt) if res else None
    y = tw.dropout(x, p, SEED, OFFSET, residual=r, out_dtype=yt)
    rows = sorted({0, 1, M // 2, M - 1} & set(range(M)))[: 1 + 16384 // d]
    keep = O.keep_mask(M, d, p, SEED, OFFSET, rows)
    xr = host(x)[rows]
    rr = None if r is None else host(r)[rows]
    want = O.dropout(xr, p, SEED, OFFSET, rr, keep)
    close(host(y)[rows], want, half_step(yt, want) * (1 + 2**-8) + 3 * U * (np.abs(xr) * 10 + (0 if rr is None else abs(rr))),
          "y")
    if r is None and p > 0:  # dropped: exact zeros; all rows: the rate
        assert np.array_equal(host(y)[rows] == 0, ~keep | (xr == 0))
        n = M * d
        assert abs(int((host(y) == 0).sum()) - p * n) <= 6 * np.sqrt(n * p * (1 - p)) + 1
    if p == 0:
        assert torch.equal(y, x.to(yt))
    # the same mask again, as a gradient's; another offset gives another
    g = tw.dropout(torch.ones_like(x), p, SEED, OFFSET)
    if r is None:
        assert torch.equal((y != 0) | (x == 0), (g != 0) | (x == 0))
    if p > 0 and M * d > 200:
        assert not torch.equal(g, tw.dropout(torch.ones_like(x), p, SEED, OFFSET + (1 << 32)))
        assert not torch.equal(g, tw.dropout(torch.ones_like(x), p, SEED + (1 << 32), OFFSET))


def test_dropout_values_in_place_and_ends():
    x = torch.full((33, 77), float("inf"), device=DEV)
    x[::2] = float("nan")
    keep = torch.from_numpy(O.keep_mask(33, 77, 0.4, 1, 0)).to(DEV)
    y = tw.dropout(x, 0.4, 1)
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()
    # x and residual written in place; nothing outside the rows is touched
    for which in ("x", "residual"):
        big = torch.arange(2 * 333 + 64, dtype=torch.float32, device=DEV)
        inner = big[32:32 + 2 * 333].view(2, 333)
        other = torch.randn(2, 333, device=DEV)
        a, b = (inner, other) if which == "x" else (other, inner)
        want = tw.dropout(a, 0.3, 5, residual=b)
        before = big.clone()
        got = tw.dropout(a, 0.3, 5, residual=b, out=inner)
        assert got.data_ptr() == inner.data_ptr() and torch.equal(inner, want)
        assert torch.equal(big[:32], before[:32]) and torch.equal(big[-32:], before[-32:])
    assert tw.dropout(torch.empty(0, 8, device=DEV), 0.5, 1).shape == (0, 8)
    assert tw.dropout(x, 0.5, (1 << 64) - 1, (1 << 64) - 1).shape == x.shape
    for bad in (-1, 1 << 64):
        with pytest.raises(ValueError):
            tw.dropout(x, 0.5, bad)
        with pytest.raises(ValueError):
            tw.dropout(x, 0.5, 1, bad)
    with pytest.raises(tw.TwellError):
        tw.dropout(x, 1.0, 1)
    with pytest.raises(ValueError):
        tw.dropout(x.t(), 0.5, 1)
    with pytest.raises(TypeError):
        tw.dropout(x.half(), 0.5, 1)
    with pytest.raises(TypeError):
        tw.dropout(x, 0.5, 1, residual=x.bfloat16(), out=torch.empty_like(x))


NORM_TYPES = [(F32, BF16, BF16, BF16, 0.1), (BF16, F32, E4M3, F32, 0.0), (F32, F32, BF16, BF16, 0.0),
              (BF16, BF16, E4M3, BF16, 0.25)]


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("xt,ht,ot,wt,p", NORM_TYPES)
def test_add_rmsnorm(M, d, xt, ht, ot, wt, p):
    print(f"[norm] {M}x{d} {xt} {ht} {ot} p={p}", flush=True)
    rng = np.random.default_rng(M * 5 + d)
    x, r, w = rand(rng, (M, d), xt), rand(rng, (M, d), ht, 2.0), rand(rng, (d,), wt)
    eps = 1e-5
    got = tw.add_rmsnorm(x, w, eps, residual=r, p=p, seed=SEED, offset=OFFSET, out_dtype=ot)
    rows = sorted({0, 1, M // 2, M - 1} & set(range(M)))[: 1 + 16384 // d]
    xr, rr, wr = host(x)[rows], host(r)[rows], host(w)
    s = O.dropout(xr, p, SEED, OFFSET, rr, O.keep_mask(M, d, p, SEED, OFFSET, rows))
    slack = 3 * U * (2 * np.abs(xr) + np.abs(rr))
    close(host(got.h)[rows], s, half_step(ht, s) * (1 + 2**-8) + slack, "h")
    n, rstd = O.rmsnorm(s, wr, eps)
    close(host(got.rstd)[rows], rstd, SUM * rstd, "rstd")
    slack = 2 * SUM * np.abs(n) + slack * rstd[:, None] * np.abs(wr)
    if ot == E4M3:
        scale = np.abs(n).max(axis=1) / 448
        close(host(got.scale)[rows], scale, 4 * SUM * scale, "scale")
        q = n / scale[:, None]
        close(host(got.n)[rows], q, half_step(ot, q) * (1 + 2**-7) + slack / scale[:, None] + 8 * SUM * np.abs(q), "n")
    else:
        assert got.scale is None
        close(host(got.n)[rows], n, half_step(ot, n) * (1 + 2**-8) + slack, "n")
    assert torch.isfinite(got.n.float()).all()  # every row was written
    # the rows that were not looked at one by one: unit mean square by the kernel's own h
    hh = host(got.h)
    r_all = 1 / np.sqrt((hh * hh).mean(axis=1) + eps)
    close(got.rstd, r_all, (2.0**-8 + SUM) * r_all, "rstd of all rows")


def test_add_rmsnorm_forms():
    """Without a residual, without h, in place, at odd addresses, twice the same."""
    rng = np.random.default_rng(3)
    for d in (333, 2048):
        x, w = rand(rng, (2100, d), BF16), rand(rng, (d,), BF16)
        a = tw.add_rmsnorm(x, w)
        assert a.h is x
        b = tw.add_rmsnorm(x, w, residual=torch.zeros_like(x))
        assert torch.equal(a.n, b.n) and torch.equal(a.rstd, b.rstd) and torch.equal(b.h, x)
        c = tw.add_rmsnorm(x, w, h_dtype=F32)
        assert torch.equal(c.h, x.float()) and torch.equal(c.n, a.n)
        drop = tw.add_rmsnorm(x, w, p=0.3, seed=4)
        assert torch.equal(drop.h, tw.dropout(x, 0.3, 4))
        r = rand(rng, (2100, d), BF16)
        want = tw.add_rmsnorm(x, w, residual=r, p=0.3, seed=4, offset=9)
        assert torch.equal(want.h, tw.dropout(x, 0.3, 4, 9, residual=r))
        again = tw.add_rmsnorm(x, w, residual=r, p=0.3, seed=4, offset=9, h=r)
        assert again.h is r
        for k in ("n", "h", "rstd"):
            assert torch.equal(getattr(want, k), getattr(again, k)), k
        # one element past an aligned base
        flat = torch.empty(5 * d + 1, dtype=BF16, device=DEV)
        odd = flat[1:].view(5, d)
        odd.copy_(x[:5])
        small = x[:5].clone()
        assert torch.equal(tw.add_rmsnorm(odd, w).n, tw.add_rmsnorm(small, w).n)
        assert torch.equal(tw.add_rmsnorm(odd, w, out_dtype=E4M3).n.view(torch.uint8),
                           tw.add_rmsnorm(small, w, out_dtype=E4M3).n.view(torch.uint8))


def test_add_rmsnorm_special_values():
    for d in (24, 1000, 5000):
        x = torch.randn(6, d, device=DEV)
        x[1] = 0
        x[2, d // 2] = float("nan")
        x[3] *= 1e-30
        x[4] *= 1e15
        w = torch.ones(d, device=DEV)
        for ot in (BF16, E4M3):
            got = tw.add_rmsnorm(x, w, 1e-6, out_dtype=ot)
            n = got.n.float()
            assert torch.isnan(n[2]).all() and torch.isnan(got.rstd[2])
            keep = [0, 1, 3, 4, 5]
            assert torch.isfinite(n[keep]).all() and (n[1] == 0).all()
            if ot == E4M3:
                assert torch.isnan(got.scale[2])
                assert (got.scale[keep] > 0).all() and torch.isfinite(got.scale[keep]).all()
                assert (n[[0, 4, 5]].abs().amax(dim=1) == 448).all()
        # eps = 0: a zero row has no direction; the other rows are as ever
        z = tw.add_rmsnorm(x, w, 0.0)
        assert torch.isnan(z.n[1].float()).all() and torch.isfinite(z.n[[0, 4, 5]].float()).all()


BWD_TYPES = [(F32, BF16, BF16, BF16, 0.1, True), (BF16, F32, F32, F32, 0.0, False), (BF16, BF16, F32, BF16, 0.0, True),
             (F32, F32, BF16, F32, 0.5, True)]


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("gt,ht,xt,wt,p,has_dh", BWD_TYPES)
def test_add_rmsnorm_backward(M, d, gt, ht, xt, wt, p, has_dh):
    print(f"[norm backward] {M}x{d} {gt} {ht} {xt} p={p}", flush=True)
    rng = np.random.default_rng(M * 3 + d)
    dn, h, w = rand(rng, (M, d), gt), rand(rng, (M, d), ht, 2.0), rand(rng, (d,), wt)
    dh = rand(rng, (M, d), ht) if has_dh else None
    rstd = tw.add_rmsnorm(h, w, 1e-5).rstd
    dres, dx, dw = tw.add_rmsnorm_backward(dn, h, w, rstd, dh=dh, p=p, seed=SEED, offset=OFFSET, dx_dtype=xt)
    dn_, h_, w_, r_ = host(dn), host(h), host(w), host(rstd)
    want, want_w = O.rmsnorm_backward(dn_, h_, w_, r_)
    g, xh = np.abs(dn_ * w_), np.abs(h_) * r_[:, None]
    mag = r_[:, None] * (g + xh * (g * xh).mean(axis=1)[:, None])
    if has_dh:
        want, mag = want + host(dh), mag + np.abs(host(dh))
    close(dres, want, half_step(ht, want) * (1 + 2**-8) + SUM * mag, "dres")
    close(dw, want_w, 256 * U * np.abs(dn_ * xh).sum(axis=0), "dweight")
    rows = sorted({0, 1, M // 2, M - 1} & set(range(M)))[: 1 + 16384 // d]
    keep = O.keep_mask(M, d, p, SEED, OFFSET, rows)
    wx = O.dropout(want[rows], p, SEED, OFFSET, keep=keep)
    close(host(dx)[rows], wx, half_step(xt, wx) * (1 + 2**-8) + 2 * SUM * mag[rows], "dx")
    if p == 0 and xt == ht:
        assert dx is dres
    again = tw.add_rmsnorm_backward(dn, h, w, rstd, dh=dh, p=p, seed=SEED, offset=OFFSET, dx_dtype=xt)
    for a, b in zip((dres, dx, dw), again):
        assert torch.equal(a, b)


def test_backward_against_differences():
    """The kernels' forward, differenced in fp32 along random directions, against the kernels' gradient."""
    rng = np.random.default_rng(11)
    M, d, eps, t = 40, 96, 1e-3, 2.0**-6
    x, r, w = (rand(rng, s, F32) for s in ((M, d), (M, d), (d,)))
    gn, gh = rand(rng, (M, d), F32), rand(rng, (M, d), F32)
    drop = dict(p=0.25, seed=SEED, offset=OFFSET)

    def norm(a, b, c):  # fp32 n from rstd and h: the kernel's n is rounded to bf16
        f = tw.add_rmsnorm(a, c, eps, residual=b, **drop)
        n = f.h.double() * f.rstd.double()[:, None] * c.double()
        return (n * gn.double()).sum() + (f.h.double() * gh.double()).sum()

    f = tw.add_rmsnorm(x, w, eps, residual=r, **drop)
    dres, dx, dw = tw.add_rmsnorm_backward(gn, f.h, w, f.rstd, dh=gh, dx_dtype=F32, **drop)
    for i, grad in ((0, dx), (1, dres), (2, dw)):
        u = rand(rng, grad.shape, F32)
        at = [x, r, w]
        # fourth order: (8 (f(t) - f(-t)) - (f(2t) - f(-2t))) / 12 t, error of order t^4 = 6e-8
        val = {k: norm(*[v + k * t * u if j == i else v for j, v in enumerate(at)]) for k in (-2, -1, 1, 2)}
        diff = float((8 * (val[1] - val[-1]) - (val[2] - val[-2])) / (12 * t))
        want = float((grad.double() * u.double()).sum())
        assert abs(diff - want) <= 1e-4 * float((grad.double() * u.double()).abs().sum()), i


def test_backward_without_rows_and_refusals():
    w = torch.ones(40, device=DEV)
    e = torch.empty(0, 40, device=DEV)
    dres, dx, dw = tw.add_rmsnorm_backward(e, e, w, torch.empty(0, device=DEV))
    assert dres.shape == (0, 40) and (dw == 0).all()
    assert tw.add_rmsnorm(e, w).n.shape == (0, 40)
    x = torch.ones(4, 40, device=DEV)
    with pytest.raises(ValueError):
        tw.add_rmsnorm(x, w[:39])
    with pytest.raises(TypeError):
        tw.add_rmsnorm(x, w, residual=x.bfloat16(), h=torch.empty_like(x))
    with pytest.raises(TypeError):
        tw.add_rmsnorm(x, w, out_dtype=F32)
    with pytest.raises(tw.TwellError):
        tw.add_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(tw.TwellError):
        tw.add_rmsnorm(torch.ones(1, 16385, device=DEV), torch.ones(16385, device=DEV))
    with pytest.raises(TypeError):
        tw.add_rmsnorm_backward(x, x, w, torch.ones(4, device=DEV), dh=x.bfloat16())


# ------------------------------------------------------------------ 4-bit products
def q4_case(rng, N, K, group, zeros, outliers=False):
    G = -(-K // group)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    z = rng.integers(0, 16, (N, G)).astype(np.uint8) if zeros else None
    s = torch.from_numpy((rng.random((N, G)) + 0.5).astype(np.float32) / (5 * K**0.5)).to(BF16)
    if outliers:  # one large weight leaves the rest of its group at zero
        q[:, :group] = 8 if z is None else z[:, :1]
        q[:, 0] = 0
        s[:, 0] = 0.3
    codes = O.pack_codes(q)
    if K % 2:
        codes[:, -1] |= (rng.integers(0, 16, N) << 4).astype(np.uint8)  # what pads a row means nothing
    W = tw.Q4(torch.from_numpy(codes).to(DEV), s.to(DEV), None if z is None else torch.from_numpy(z).to(DEV), K, group)
    return W, O.q4_dequantize(q, s.double().numpy(), z, group)


def q4_x(rng, M, K, xt):
    if xt != E4M3:
        x = rand(rng, (M, K), xt)
        return x, None, host(x)
    x = rand(rng, (M, K), F32, 40.0).to(E4M3)
    sx = rand(rng, (M,), F32).abs() / 40
    return x, sx, host(x) * host(sx)[:, None]


Q4_SIZES = [  # M, N, K, group
    (1, 1, 1, 32), (1, 16, 32, 32), (2, 17, 33, 32), (3, 5, 127, 64), (5, 100, 129, 128), (1, 64, 2048, 128),
    (16, 40, 1100, 64), (17, 33, 640, 32), (33, 130, 257, 128), (64, 48, 1024, 64), (65, 31, 515, 32),
    (130, 257, 383, 64), (256, 96, 256, 128), (4, 2051, 96, 32), (300, 129, 4100, 128), (1, 24, 10240, 64)]


@pytest.mark.parametrize("M,N,K,group", Q4_SIZES)
@pytest.mark.parametrize("xt,yt,zeros", [(BF16, F32, False), (F32, F32, True), (E4M3, BF16, False), (BF16, BF16, True),
                                         (E4M3, F32, True), (F32, F32, False)])
def test_q4_matmul(M, N, K, group, xt, yt, zeros):
    print(f"[q4] {M}x{N}x{K} group {group} {xt} {yt} zeros {zeros}", flush=True)
    rng = np.random.default_rng(M + N + K)
    W, w = q4_case(rng, N, K, group, zeros)
    x, sx, xv = q4_x(rng, M, K, xt)
    big = torch.full((M * N + 128,), 7.0, dtype=yt, device=DEV)
    y = tw.q4_matmul(x, W, x_scale=sx, y=big[64:64 + M * N].view(M, N))
    want = xv @ w.T
    close(y, want, half_step(yt, want) * (1 + 2**-8) + (K + 512) * U * (np.abs(xv) @ np.abs(w).T), "y")
    assert (big[:64] == 7).all() and (big[-64:] == 7).all()
    assert torch.equal(y, tw.q4_matmul(x, W, x_scale=sx, out_dtype=yt))


# Sizes that take other tiles and splits than the ones above: 128 rows a
# workgroup, K in many parts, two waves side by side for few rows.
@pytest.mark.parametrize("M,N,K,group", [(259, 8200, 645, 64), (385, 8193, 128, 32), (513, 70, 2100, 128), (5, 4201, 300, 32),
                                         (3, 2051, 8300, 128), (16, 4100, 2049, 64), (129, 300, 4104, 64)])
@pytest.mark.parametrize("xt,yt,zeros", [(BF16, F32, True), (F32, BF16, False), (E4M3, F32, True)])
def test_q4_matmul_other_tiles(M, N, K, group, xt, yt, zeros):
    test_q4_matmul(M, N, K, group, xt, yt, zeros)


# Enough rows and units for the kernel of large products: cut K, K in parts, the
# tiles of each number of rows.
@pytest.mark.parametrize("M,N,K,group", [(40, 8200, 1100, 32), (33, 8193, 1027, 64), (70, 5000, 2101, 64), (130, 1100, 8200, 128),
                                         (200, 4100, 96, 32), (65, 8200, 513, 128)])
@pytest.mark.parametrize("xt,yt,zeros", [(BF16, F32, True), (F32, BF16, False), (E4M3, F32, True)])
def test_q4_matmul_large(M, N, K, group, xt, yt, zeros):
    test_q4_matmul(M, N, K, group, xt, yt, zeros)


@pytest.mark.parametrize("M,F,d,group", [(1, 1024, 256, 128), (3, 77, 300, 32), (16, 130, 513, 64), (70, 200, 129, 32),
                                         (40, 64, 2560, 128)])
@pytest.mark.parametrize("xt,zeros", [(BF16, False), (E4M3, True), (F32, False)])
def test_q4_gateup_and_ffn(M, F, d, group, xt, zeros):
    print(f"[q4 ffn] {M} rows d={d} F={F} group {group} {xt} zeros {zeros}", flush=True)
    rng = np.random.default_rng(M + F + d)
    (Wg, wg), (Wu, wu), (Wd, wd) = (q4_case(rng, F, d, group, zeros, True), q4_case(rng, F, d, group, zeros),
                                    q4_case(rng, d, F, group, zeros))
    x, sx, xv = q4_x(rng, M, d, xt)
    z, u = np.abs(xv) @ np.abs(wg).T, np.abs(xv) @ np.abs(wu).T  # magnitudes for the bounds
    want = O.gated_hidden(xv, wg, wu)
    b = (d + 512) * U
    slack = b * (z * np.abs(xv @ wu.T) + u * np.abs(xv @ wg.T)) + b * b * z * u
    for ht in (F32, BF16):
        h = tw.q4_gateup(x, Wg, Wu, x_scale=sx, out_dtype=ht)
        close(h, want, half_step(ht, want) * (1 + 2**-7) + slack, "h")
    y = tw.ffn_forward_q4(x, Wg, Wu, Wd, x_scale=sx)
    assert y.dtype == F32
    close(y, want @ wd.T, (slack + U * np.abs(want)) @ np.abs(wd).T + (F + 512) * U * (np.abs(want) @ np.abs(wd).T), "y")
    assert torch.equal(y, tw.ffn_forward_q4(x, Wg, Wu, Wd, x_scale=sx))


@pytest.mark.parametrize("M,F,d,group", [(260, 4100, 200, 64), (385, 2100, 136, 32), (9, 600, 4500, 128)])
@pytest.mark.parametrize("xt,zeros", [(BF16, True), (E4M3, False), (F32, True)])
def test_q4_gateup_and_ffn_other_tiles(M, F, d, group, xt, zeros):
    test_q4_gateup_and_ffn(M, F, d, group, xt, zeros)


@pytest.mark.parametrize("M,F,d,group", [(40, 8200, 300, 32), (70, 3001, 1030, 64), (20, 8300, 520, 128)])
@pytest.mark.parametrize("xt,zeros", [(BF16, True), (E4M3, False), (F32, True)])
def test_q4_gateup_and_ffn_large(M, F, d, group, xt, zeros):
    test_q4_gateup_and_ffn(M, F, d, group, xt, zeros)


def test_q4_large_weight_in_a_group():
    """A group of one large weight and zeros: nothing large may cancel (8 x sums of 128
    terms would leave 2^-24 * 8 * 128 * 0.3 = 2e-5 where 1e-6 is the bound)."""
    rng = np.random.default_rng(8)
    for xt in (BF16, E4M3, F32):
        for zeros in (False, True):
            W, w = q4_case(rng, 64, 256, 128, zeros, outliers=True)
            x, sx, xv = q4_x(rng, 4, 256, xt)
            xv[:, 0] = 0
            x[:, 0] = 0
            want = xv @ w.T
            close(tw.q4_matmul(x, W, x_scale=sx), want, 256 * U * (np.abs(xv) @ np.abs(w).T), "y")


def test_q4_rows_do_not_mix():
    """An infinity or NaN in one row of x stays in that row; a NaN gate is not active."""
    rng = np.random.default_rng(9)
    for M in (3, 20, 80):
        W, w = q4_case(rng, 50, 200, 64, False)
        x = rand(rng, (M, 200), BF16)
        clean = tw.q4_matmul(x, W)
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        y = tw.q4_matmul(x, W)
        rows = [0] + list(range(3, M))
        assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
        h = tw.q4_gateup(x, W, W)
        assert (h[1] == 0).all()


@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (5, 31, 32), (33, 200, 64), (64, 1025, 128), (300, 256, 32)])
def test_q4_quantize(N, K, group):
    rng = np.random.default_rng(N + K)
    W = rand(rng, (N, K), BF16)
    W[0, : min(K, group)] = 0
    if N > 4:
        W[4] *= 1e-20
    q = tw.q4_quantize(W, group)
    codes, scales = O.q4_quantize(host(W), group)
    assert np.array_equal(host(q.scales), scales)
    mask = np.full(codes.shape[1] + codes.shape[1] % 2, 15, dtype=np.uint8)
    if K % 2:
        mask[-1] = 0  # what pads a row
    mask = mask[0::2] | (mask[1::2] << 4)
    assert np.array_equal(q.codes.cpu().numpy() & mask, O.pack_codes(codes) & mask)
    x = rand(rng, (2, K), BF16)
    w = O.q4_dequantize(codes, scales, None, group)
    want = host(x) @ w.T
    close(tw.q4_matmul(x, q), want, (K + 512) * U * (np.abs(host(x)) @ np.abs(w).T), "y")


def test_q4_binding_refusals():
    rng = np.random.default_rng(2)
    W, _ = q4_case(rng, 32, 64, 32, True)
    x = rand(rng, (4, 64), BF16)
    with pytest.raises(ValueError):
        tw.q4_matmul(x[:, :63].contiguous(), W)
    with pytest.raises(ValueError):
        tw.q4_matmul(x.t(), W)
    with pytest.raises(ValueError):
        tw.q4_matmul(x, W, x_scale=torch.ones(4, device=DEV))
    with pytest.raises(ValueError):
        tw.q4_matmul(x.to(E4M3), W)
    with pytest.raises(TypeError):
        tw.q4_matmul(x.half(), W)
    with pytest.raises(ValueError):
        tw.q4_matmul(x, tw.Q4(W.codes, W.scales[:, :1].contiguous(), W.zeros, 64, 32))
    with pytest.raises(ValueError):
        tw.q4_matmul(x, tw.Q4(W.codes, W.scales, W.zeros.cpu(), 64, 32))
    with pytest.raises(tw.TwellError):
        tw.q4_quantize(rand(rng, (4, 64), BF16), 48)
    V, _ = q4_case(rng, 32, 64, 64, True)
    with pytest.raises(ValueError):
        tw.q4_gateup(x, W, V)  # groups differ
    assert tw.q4_matmul(x[:0], W).shape == (0, 32)
    assert tw.ffn_forward_q4(x[:0], W, W, q4_case(rng, 64, 32, 32, False)[0]).shape == (0, 64)


# ------------------------------------------------------------------ as they are used
def test_side_stream_and_graph():
    """A serving block on a stream of its own and in a graph: the eager bits, every replay."""
    rng = np.random.default_rng(21)
    M, d, F = 4, 256, 512
    (Wg, _), (Wu, _), (Wd, _) = (q4_case(rng, F, d, 64, False), q4_case(rng, F, d, 64, True), q4_case(rng, d, F, 64, False))
    w = rand(rng, (d,), BF16)
    x, res = rand(rng, (M, d), F32), rand(rng, (M, d), BF16)

    def block(x, res):
        n = tw.add_rmsnorm(x, w, residual=res, out_dtype=E4M3)
        y = tw.ffn_forward_q4(n.n, Wg, Wu, Wd, x_scale=n.scale)
        return y, tw.add_rmsnorm(y, w, residual=n.h, p=0.1, seed=3).n

    want = block(x, res)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = block(x, res)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    gx, gr = x.clone(), res.clone()
    with torch.cuda.graph(graph):
        out = block(gx, gr)
    for k in range(4):
        nx = rand(np.random.default_rng(100 + k), (M, d), F32)
        gx.copy_(nx)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(block(nx, res), out):
            assert torch.equal(a, b), k
