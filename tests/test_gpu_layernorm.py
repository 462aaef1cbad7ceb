"""Layer norm and its backward on the GPU, through the binding, against the fp64
oracle at the sizes, types and values where they can go wrong.

Error bounds, u = 2^-24, derived from the arithmetic:
* s = residual + x k: at most 3 u (2 |x| + |r|) off (k and the product, the sum), e_s below.
* The mean is a sum of chains of at most 16 + 6 + 16 terms, taken twice (around the
  rounded mean): off by e_s plus 4 u of the row's largest |s|; e below.
* A deviation is off by e + u |c|, the variance by twice their relative size (root mean
  square over the deviations) and SUM = 2^-17 for the sums of squares (128 u; the longest
  chain is 16 terms a thread, 6 levels, 16 waves), rstd by half of that.
* out = c rstd w + b: the parts' errors and 4 u of each magnitude; bf16 2^-8 of
  the value on top, e4m3 2^-4 of it, at least 2^-10.
* Backward: two sums of 38-term chains, 2^-17 of the sum of magnitudes each; dw and db at
  most M / 512 rows a workgroup, 4 waves, 16 + 5 additions: under 256 u for the sizes here."""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, OFFSET, SEED, SIZES, SUM, U, close, half_step, host, rand  # noqa: E402


def bounds(s, e_s, w, b, eps):
    """(n, mean, rstd, bound of mean, relative bound of rstd, bound of n before it is rounded)."""
    n, mean, rstd = O.layernorm(s, w, b, eps)
    e = e_s + 4 * U * np.abs(s).max(axis=1, keepdims=True)
    c = s - mean[:, None]
    off = np.sqrt(((e + U * np.abs(c)) ** 2).mean(axis=1)) * rstd  # of a deviation, against the root of the variance
    rel = SUM + off + off * off + 4 * U
    hat = np.abs(c) * rstd[:, None]
    slack = (e * rstd[:, None] + hat * rel[:, None] + 4 * U * hat) * np.abs(w) + 4 * U * (
        np.abs(hat * w) + (0 if b is None else np.abs(b)))
    return n, mean, rstd, e.max(axis=1), rel, slack


def check(got, rows, s, e_s, w, b, eps, ot, ht):
    close(host(got.h)[rows], s, half_step(ht, s) * (1 + 2**-8) + e_s, "h")
    n, mean, rstd, e_mean, rel, slack = bounds(s, e_s, w, b, eps)
    close(host(got.mean)[rows], mean, e_mean + U * np.abs(mean), "mean")
    close(host(got.rstd)[rows], rstd, rel * rstd, "rstd")
    if ot == BF16:
        assert got.scale is None
        close(host(got.n)[rows], n, half_step(ot, n) * (1 + 2**-8) + slack, "n")
        return
    scale = np.maximum(np.abs(n).max(axis=1), 2.0**-100) / 448
    e_scale = slack.max(axis=1) / 448 + 2 * U * scale
    close(host(got.scale)[rows], scale, e_scale, "scale")
    q = n / scale[:, None]
    rel_scale = (e_scale / scale)[:, None]
    close(host(got.n)[rows], q, half_step(ot, q) * (1 + 2**-6) + (slack / scale[:, None] + (rel_scale + 4 * U) * np.abs(q)) * (1 + 2**-4),
          "n")


TYPES = [(F32, BF16, BF16, BF16, 0.1, True), (BF16, F32, E4M3, F32, 0.0, False), (F32, F32, BF16, BF16, 0.0, True),
         (BF16, BF16, E4M3, BF16, 0.25, True)]


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("xt,ht,ot,wt,p,has_bias", TYPES)
def test_add_layernorm(M, d, xt, ht, ot, wt, p, has_bias):
    print(f"[layernorm] {M}x{d} {xt} {ht} {ot} p={p}", flush=True)
    rng = np.random.default_rng(M * 5 + d)
    x, r, w = rand(rng, (M, d), xt), (rand(rng, (M, d), F32, 2.0) + 0.75).to(ht), rand(rng, (d,), wt)
    b = rand(rng, (d,), wt) if has_bias else None
    eps = 1e-5
    got = tw.add_layernorm(x, w, b, eps, residual=r, p=p, seed=SEED, offset=OFFSET, out_dtype=ot)
    rows = sorted({0, 1, M // 2, M - 1} & set(range(M)))[: 1 + 16384 // d]
    xr, rr = host(x)[rows], host(r)[rows]
    s = O.dropout(xr, p, SEED, OFFSET, rr, O.keep_mask(M, d, p, SEED, OFFSET, rows))
    check(got, rows, s, 3 * U * (2 * np.abs(xr) + np.abs(rr)), host(w), None if b is None else host(b), eps, ot, ht)
    assert torch.isfinite(got.n.float()).all()  # every row was written
    # the rows that were not looked at one by one: by the kernel's own h, each element of which is
    # half a step off
    hh = host(got.h)
    close(got.mean, hh.mean(axis=1), (half_step(ht, hh) * 2).max(axis=1) + 4 * U * np.abs(hh).max(axis=1), "mean of all rows")
    again = tw.add_layernorm(x, w, b, eps, residual=r, p=p, seed=SEED, offset=OFFSET, out_dtype=ot)
    assert torch.equal(got.n.view(torch.uint8), again.n.view(torch.uint8)) and torch.equal(got.rstd, again.rstd)


def test_forms():
    """Without a residual, without h, in place, at odd addresses."""
    rng = np.random.default_rng(3)
    for d in (333, 2048):
        x, w, b = rand(rng, (2100, d), BF16), rand(rng, (d,), BF16), rand(rng, (d,), BF16)
        a = tw.add_layernorm(x, w, b)
        assert a.h is x
        z = tw.add_layernorm(x, w, b, residual=torch.zeros_like(x))
        assert torch.equal(a.n, z.n) and torch.equal(a.rstd, z.rstd) and torch.equal(a.mean, z.mean) and torch.equal(z.h, x)
        assert torch.equal(tw.add_layernorm(x, w, torch.zeros_like(b)).n, tw.add_layernorm(x, w).n)
        c = tw.add_layernorm(x, w, b, h_dtype=F32)
        assert torch.equal(c.h, x.float()) and torch.equal(c.n, a.n)
        drop = tw.add_layernorm(x, w, b, p=0.3, seed=4)
        assert torch.equal(drop.h, tw.dropout(x, 0.3, 4))
        r = rand(rng, (2100, d), BF16)
        want = tw.add_layernorm(x, w, b, residual=r, p=0.3, seed=4, offset=9)
        assert torch.equal(want.h, tw.dropout(x, 0.3, 4, 9, residual=r))
        again = tw.add_layernorm(x, w, b, residual=r, p=0.3, seed=4, offset=9, h=r)
        assert again.h is r
        for k in ("n", "h", "mean", "rstd"):
            assert torch.equal(getattr(want, k), getattr(again, k)), k
        # one element past an aligned base
        flat = torch.empty(5 * d + 1, dtype=BF16, device=DEV)
        odd = flat[1:].view(5, d)
        odd.copy_(x[:5])
        small = x[:5].clone()
        for ot in (BF16, E4M3):
            assert torch.equal(tw.add_layernorm(odd, w, b, out_dtype=ot).n.view(torch.uint8),
                               tw.add_layernorm(small, w, b, out_dtype=ot).n.view(torch.uint8))


@pytest.mark.parametrize("d", [24, 512, 1000, 5000, 12001])
def test_rows_with_a_large_mean(d):
    """The variance is not a difference of large sums: a mean 4096 deviations away."""
    print(f"[layernorm mean] {d}", flush=True)
    rng = np.random.default_rng(d)
    x = rand(rng, (5, d), F32) + 4096.0 * torch.tensor([[1.0], [-1.0], [1.0], [0.5], [0.0]], device=DEV)
    w, b = rand(rng, (d,), F32), rand(rng, (d,), F32)
    s = host(x)
    for ot in (BF16, E4M3):
        check(tw.add_layernorm(x, w, b, 1e-5, residual=torch.zeros_like(x), out_dtype=ot), list(range(5)), s,
              np.zeros_like(s), host(w), host(b), 1e-5, ot, F32)


@pytest.mark.parametrize("d", [24, 512, 1000, 5000, 12001])
@pytest.mark.parametrize("ht", [F32, BF16])
@pytest.mark.parametrize("eps", [0.0, 1e-5, 1e-35])
def test_rows_over_the_range(d, ht, eps):
    """Rows whose squares pass fp32's range in either direction, and those whose sum does.
    What lies under 2^-126 has steps of 2^-149: a deviation of a row of 2^-120 is
    that much off, and so is the rstd of the largest rows."""
    print(f"[layernorm range] {d} {ht} {eps}", flush=True)
    rng = np.random.default_rng(d)
    powers = (-110, -100, -75, -65, -50, 0, 40, 58, 60, 62, 64, 100, 124)
    x = torch.stack([rand(rng, (d,), F32).clamp(-7, 7) * 2.0**e for e in powers]).to(ht)
    w = rand(rng, (d,), BF16)
    s, wr = host(x), host(w)
    n, mean, rstd, e_mean, rel, slack = bounds(s, np.zeros_like(s) + 2.0**-149, wr, None, float(np.float32(eps)))
    for ot in (BF16, E4M3):
        got = tw.add_layernorm(x, w, None, eps, residual=torch.zeros_like(x), out_dtype=ot)
        assert torch.equal(got.h, x)
        close(got.mean, mean, e_mean + U * np.abs(mean) + 2.0**-148, "mean")
        close(got.rstd, rstd, rel * rstd + 2.0**-149, "rstd")
        if ot == BF16:
            close(got.n, n, half_step(BF16, n) * (1 + 2**-8) + slack + 2.0**-133, "n")  # bf16's least step
            continue
        scale = np.maximum(np.abs(n).max(axis=1), 2.0**-100) / 448
        e_scale = slack.max(axis=1) / 448 + 2 * U * scale
        close(got.scale, scale, e_scale, "scale")
        q = n / scale[:, None]
        close(got.n, q, half_step(E4M3, q) * (1 + 2**-6) + (slack / scale[:, None] + ((e_scale / scale)[:, None] + 4 * U) * np.abs(q)) * (1 + 2**-4),
              "n")


def test_special_values():
    for d in (24, 1000, 5000, 9000):
        x = torch.randn(7, d, device=DEV)
        x[1] = 0
        x[2, d // 2] = float("nan")
        x[3] = 3e38  # a sum past the range
        x[4, d - 1] = float("inf")
        x[5] = torch.finfo(BF16).min
        w, b = torch.full((d,), 2.0, device=DEV), torch.full((d,), 0.5, device=DEV)
        for ot in (BF16, E4M3):
            got = tw.add_layernorm(x, w, b, 1e-5, out_dtype=ot)
            n = got.n.float()
            for row in (2, 4):
                assert torch.isnan(n[row]).all() and torch.isnan(got.rstd[row]), (d, row)
                assert ot == BF16 or torch.isnan(got.scale[row])
            for row in (1, 3, 5):  # equal values: the bias alone
                value = n[row] * (1 if ot == BF16 else got.scale[row])
                assert torch.allclose(value, b, rtol=2.0**-20, atol=0), (d, row)
                assert got.mean[row] == x[row, 0]
            assert torch.isfinite(n[[0, 6]]).all()
        z = tw.add_layernorm(x, w, b, 0.0)
        assert torch.isnan(z.n[[1, 3, 5]].float()).all() and torch.isfinite(z.n[[0, 6]].float()).all()


BWD_TYPES = [(F32, BF16, BF16, BF16, 0.1, True), (BF16, F32, F32, F32, 0.0, False), (BF16, BF16, F32, BF16, 0.0, True),
             (F32, F32, BF16, F32, 0.5, True)]


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("gt,ht,xt,wt,p,has_dh", BWD_TYPES)
def test_add_layernorm_backward(M, d, gt, ht, xt, wt, p, has_dh):
    print(f"[layernorm backward] {M}x{d} {gt} {ht} {xt} p={p}", flush=True)
    rng = np.random.default_rng(M * 3 + d)
    dn, h, w = rand(rng, (M, d), gt), (rand(rng, (M, d), F32, 2.0) + 0.75).to(ht), rand(rng, (d,), wt)
    dh = rand(rng, (M, d), ht) if has_dh else None
    f = tw.add_layernorm(h, w, None, 1e-5)
    args = dict(dh=dh, p=p, seed=SEED, offset=OFFSET, dx_dtype=xt)
    dres, dx, dw, db = tw.add_layernorm_backward(dn, h, w, f.mean, f.rstd, **args)
    dn_, h_, w_, m_, r_ = host(dn), host(h), host(w), host(f.mean), host(f.rstd)
    want, want_w, want_b = O.layernorm_backward(dn_, h_, w_, m_, r_)
    g, xh = np.abs(dn_ * w_), (np.abs(h_) + np.abs(m_)[:, None]) * r_[:, None]
    mag = r_[:, None] * (g + g.mean(axis=1, keepdims=True) + xh * (g * xh).mean(axis=1, keepdims=True))
    if has_dh:
        want, mag = want + host(dh), mag + np.abs(host(dh))
    close(dres, want, half_step(ht, want) * (1 + 2**-8) + SUM * mag, "dres")
    close(dw, want_w, 256 * U * np.abs(dn_ * xh).sum(axis=0), "dweight")
    close(db, want_b, 256 * U * np.abs(dn_).sum(axis=0), "dbias")
    rows = sorted({0, 1, M // 2, M - 1} & set(range(M)))[: 1 + 16384 // d]
    keep = O.keep_mask(M, d, p, SEED, OFFSET, rows)
    wx = O.dropout(want[rows], p, SEED, OFFSET, keep=keep)
    close(host(dx)[rows], wx, half_step(xt, wx) * (1 + 2**-8) + 2 * SUM * mag[rows], "dx")
    if p == 0 and xt == ht:
        assert dx is dres
    for a, b in zip((dres, dx, dw, db), tw.add_layernorm_backward(dn, h, w, f.mean, f.rstd, **args)):
        assert torch.equal(a, b)


def test_backward_against_differences():
    """The kernels' forward, differenced in fp32 along random directions, against the kernels' gradient."""
    rng = np.random.default_rng(11)
    M, d, eps, t = 40, 96, 1e-3, 2.0**-6
    x, r, w, b = (rand(rng, s, F32) for s in ((M, d), (M, d), (d,), (d,)))
    gn, gh = rand(rng, (M, d), F32), rand(rng, (M, d), F32)
    drop = dict(p=0.25, seed=SEED, offset=OFFSET)

    def norm(a, c, e, k):  # fp32 n from h, mean and rstd: the kernel's n is rounded to bf16
        f = tw.add_layernorm(a, e, k, eps, residual=c, **drop)
        n = (f.h.double() - f.mean.double()[:, None]) * f.rstd.double()[:, None] * e.double() + k.double()
        return (n * gn.double()).sum() + (f.h.double() * gh.double()).sum()

    f = tw.add_layernorm(x, w, b, eps, residual=r, **drop)
    dres, dx, dw, db = tw.add_layernorm_backward(gn, f.h, w, f.mean, f.rstd, dh=gh, dx_dtype=F32, **drop)
    for i, grad in ((0, dx), (1, dres), (2, dw), (3, db)):
        u = rand(rng, grad.shape, F32)
        at = [x, r, w, b]
        # fourth order: (8 (f(t) - f(-t)) - (f(2t) - f(-2t))) / 12 t, error of order t^4 = 6e-8
        val = {k: norm(*[v + k * t * u if j == i else v for j, v in enumerate(at)]) for k in (-2, -1, 1, 2)}
        diff = float((8 * (val[1] - val[-1]) - (val[2] - val[-2])) / (12 * t))
        want = float((grad.double() * u.double()).sum())
        assert abs(diff - want) <= 1e-4 * float((grad.double() * u.double()).abs().sum()), i


def test_backward_outputs_left_out_and_in_place():
    """dres or dx or dbias not asked for, dres written over dh, through the C entry."""
    import ctypes

    L = tw.lib()
    rng = np.random.default_rng(2)
    for M, d in ((70, 40), (70, 1001), (9, 9000)):
        dn, h, w, dh = rand(rng, (M, d), F32), rand(rng, (M, d), BF16), rand(rng, (d,), BF16), rand(rng, (M, d), BF16)
        f = tw.add_layernorm(h, w)
        dres, dx, dw, db = tw.add_layernorm_backward(dn, h, w, f.mean, f.rstd, dh=dh, p=0.2, seed=5, dx_dtype=F32)
        ws = tw.Workspace(DEV)
        wp, wn = ws.get(tw.layernorm_workspace_bytes(M, d))

        def run(dres_p, dx_p, db_p, dh_t):
            out = torch.empty(d, device=DEV)
            st = L.twell_add_layernorm_backward(
                dn.data_ptr(), 1, dh_t.data_ptr(), h.data_ptr(), 0, w.data_ptr(), 0, f.mean.data_ptr(), f.rstd.data_ptr(),
                M, d, 0.2, 5, 0, dres_p, dx_p, 1, out.data_ptr(), db_p, wp, wn,
                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
            assert st == 0
            assert torch.equal(out, dw)

        only = torch.empty_like(dx)
        run(None, only.data_ptr(), None, dh)
        assert torch.equal(only, dx)
        over, bias = dh.clone(), torch.empty(d, device=DEV)
        run(over.data_ptr(), None, bias.data_ptr(), over)
        assert torch.equal(over, dres) and torch.equal(bias, db)


def test_nothing_beside_the_rows_is_written():
    rng = np.random.default_rng(6)
    for M, d in ((3, 7), (5, 300), (4, 2049), (2, 9001)):
        x, w, r = rand(rng, (M, d), F32), rand(rng, (d,), F32), rand(rng, (M, d), BF16)
        big = torch.full((M * d + 64,), 7.0, device=DEV, dtype=BF16)
        h = big[32:32 + M * d].view(M, d)
        h.copy_(r)
        tw.add_layernorm(x, w, w, residual=h, h=h)
        assert (big[:32] == 7).all() and (big[-32:] == 7).all()


def test_no_rows_and_refusals():
    w = torch.ones(40, device=DEV)
    e, none = torch.empty(0, 40, device=DEV), torch.empty(0, device=DEV)
    dres, dx, dw, db = tw.add_layernorm_backward(e, e, w, none, none)
    assert dres.shape == (0, 40) and (dw == 0).all() and (db == 0).all()
    assert tw.add_layernorm(e, w).n.shape == (0, 40)
    x = torch.ones(4, 40, device=DEV)
    for bad in (lambda: tw.add_layernorm(x, w[:39]), lambda: tw.add_layernorm(x, w, w[:39]), lambda: tw.add_layernorm(x.t(), w),
                lambda: tw.add_layernorm(x, w, seed=-1), lambda: tw.add_layernorm_backward(x, x, w, w[:3], w[:4])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tw.add_layernorm(x, w, w.bfloat16()), lambda: tw.add_layernorm(x, w, out_dtype=F32),
                lambda: tw.add_layernorm(x, w, residual=x.bfloat16(), h=torch.empty_like(x)),
                lambda: tw.add_layernorm_backward(x, x, w, w[:4], w[:4], dh=x.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(tw.TwellError):
        tw.add_layernorm(x, w, eps=-1.0)
    with pytest.raises(tw.TwellError):
        tw.add_layernorm(torch.ones(1, 16385, device=DEV), torch.ones(16385, device=DEV))


@pytest.mark.parametrize("M,d", [((1 << 23) + 5, 8), ((1 << 21) + 3, 513)])
def test_more_rows_than_one_dimension_of_a_launch(M, d):
    print(f"[layernorm rows] {M}x{d}", flush=True)
    edge = 1 << 21
    rows = sorted({0, 1, 4 * edge - 1, 4 * edge, 4 * edge + 1, edge - 1, edge, edge + 1, M - 2, M - 1} & set(range(M)))
    rng = np.random.default_rng(d)
    at = torch.tensor(rows, device=DEV)
    x = torch.empty(M, d, dtype=BF16, device=DEV).fill_(0.5)
    x[at] = rand(rng, (len(rows), d), BF16)
    w, b = rand(rng, (d,), BF16), rand(rng, (d,), BF16)
    r = tw.add_layernorm(x, w, b, 1e-5)
    n, mean, rstd, e_mean, rel, slack = bounds(host(x[at]), np.zeros((len(rows), d)), host(w), host(b), 1e-5)
    close(host(r.n[at]), n, half_step(BF16, n) * (1 + 2**-8) + slack, "n")
    close(host(r.rstd[at]), rstd, rel * rstd, "rstd")
    other = torch.ones(M, dtype=torch.bool, device=DEV)
    other[at] = False
    assert (r.mean[other] == 0.5).all()
    for i in range(0, M, 1 << 20):
        assert bool((r.n[i:i + (1 << 20)] == b).all(dim=1)[other[i:i + (1 << 20)]].all()), i
    # the backward's dbias meets every row once
    ones = torch.ones(M, d, dtype=BF16, device=DEV)
    _, _, _, db = tw.add_layernorm_backward(ones, x, w, r.mean, r.rstd)
    assert (db == M).all()  # whole numbers below 2^24


@pytest.mark.parametrize("M,d", [(70001, 250), (17000, 1001), (8301, 2049), (2101, 8193)])
def test_outputs_past_the_l2(M, d):
    """Outputs of 32 MB and more are stored another way: the same bits as in parts that are smaller."""
    print(f"[layernorm large] {M}x{d}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r, dn = (torch.randn((M, d), generator=g, device=DEV) for _ in range(3))
    r = r.to(BF16)
    w, b = torch.randn(d, generator=g, device=DEV), torch.randn(d, generator=g, device=DEV)
    got = tw.add_layernorm(x, w, b, residual=r)
    dres, dx, dw, db = tw.add_layernorm_backward(dn, got.h, w, got.mean, got.rstd, dh=r, dx_dtype=F32)
    part = M // 7 + 1
    for i in range(0, M, part):
        at = slice(i, i + part)
        few = tw.add_layernorm(x[at], w, b, residual=r[at])
        for k in ("n", "h", "mean", "rstd"):
            assert torch.equal(getattr(got, k)[at], getattr(few, k)), (i, k)
        back = tw.add_layernorm_backward(dn[at], few.h, w, few.mean, few.rstd, dh=r[at], dx_dtype=F32)
        assert torch.equal(back[0], dres[at]) and torch.equal(back[1], dx[at]), i


def test_captured_and_replayed():
    """A graph of both calls, replayed with eager work between; and two streams at once."""
    rng = np.random.default_rng(8)
    M, d = 300, 2048
    x, r, w, b, dn = (rand(rng, s, F32) for s in ((M, d), (M, d), (d,), (d,), (M, d)))

    def both():
        f = tw.add_layernorm(x, w, b, residual=r, p=0.1, seed=3)
        return (f.n, f.h, *tw.add_layernorm_backward(dn, f.h, w, f.mean, f.rstd, p=0.1, seed=3))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(4):
        x.copy_(rand(rng, (M, d), F32))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), k
    want = both()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(both())
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))
