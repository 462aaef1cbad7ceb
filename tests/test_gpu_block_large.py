"""Operators around the FFN at sizes of memory: rows past what one dimension of a
launch holds, outputs that are stored past the L2 (32 MB and more), offsets past 32
bits. Against the fp64 oracle, with the bounds of tests/test_gpu_block.py's kind:
2^-8 of a bf16 value and 2^-4 of an e4m3 one (or 2^-10), fp32 sums 2^-17 of their
magnitude, dweight M / 512 + 64 additions, 4-bit products K + 512."""

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
SEED, OFFSET = 0x0FEDCBA987654321, (3 << 32) + 11


def host(t):
    return t.double().cpu().numpy()


def half_step(dtype, v):
    """Largest rounding of v to dtype."""
    if dtype == F32:
        return U * np.abs(v)
    return 2.0**-8 * np.abs(v) if dtype == BF16 else np.maximum(2.0**-4 * np.abs(v), 2.0**-10)


def close(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound + 1e-37)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def room(gib):
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < (gib + 4) << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


# (8 columns: a wave a row, four rows a workgroup; 2^24 rows of 1537 or more take a
# workgroup of 256 threads each)
@pytest.mark.parametrize("M,d,gib", [((1 << 23) + 5, 8, 1), ((1 << 21) + 3, 513, 4), (1 << 24, 1537, 76)])
def test_norm_of_many_rows(M, d, gib):
    print(f"[large] norm of {M} rows of {d}", flush=True)
    room(gib)
    edge = 1 << 21
    rows = sorted({0, 1, 4 * edge - 1, 4 * edge, 4 * edge + 1, edge - 1, edge, edge + 1, M - 2, M - 1} & set(range(M)))
    rng = np.random.default_rng(d)
    at = torch.tensor(rows, device=DEV)
    x = torch.empty(M, d, dtype=BF16, device=DEV).fill_(0.5)
    x[at] = torch.from_numpy(rng.standard_normal((len(rows), d)).astype(np.float32)).to(BF16).to(DEV)
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(BF16).to(DEV)
    r = tw.add_rmsnorm(x, w, 1e-5, out_dtype=E4M3)
    n, rstd = O.rmsnorm(host(x[at]), host(w), 1e-5)
    close(host(r.rstd[at]), rstd, SUM * rstd, "rstd")
    scale = np.abs(n).max(axis=1) / 448
    close(host(r.scale[at]), scale, 4 * SUM * scale, "scale")
    q = n / scale[:, None]
    close(host(r.n[at].float()), q, half_step(E4M3, q) * (1 + 2**-7) + 16 * SUM * np.abs(q), "n")
    # all rows but those are alike, and every one was written
    other = torch.ones(M, dtype=torch.bool, device=DEV)
    other[at] = False
    assert (r.rstd[other] == r.rstd[2]).all() and (r.scale[other] == r.scale[2]).all()
    for i in range(0, M, 1 << 20):
        part = r.n[i:i + (1 << 20)].view(torch.uint8)
        assert bool((part == r.n[2].view(torch.uint8)).all(dim=1)[other[i:i + (1 << 20)]].all()), i


# ------------------------------------------------------------------ outputs past the L2
def normal(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(dtype)


def guarded(M, d, dtype):
    """An [M, d] tensor inside a larger one: (whole, inner, check)."""
    big = torch.full((M * d + 128,), 7.0, device=DEV).to(dtype)

    def check():
        assert (big[:64] == 7).all() and (big[-64:] == 7).all()

    return big[64:64 + M * d].view(M, d), check


# a wave a row, then workgroups of 2 to 16 waves with one or two blocks a thread; whole and
# cut rows, whose stores are at every address
LARGE = [(70001, 250), (70001, 256), (17000, 1001), (8300, 2048), (8301, 2049), (2101, 8193), (2100, 8192), (1101, 16383),
         (4111, 5003)]


@pytest.mark.parametrize("M,d", LARGE)
@pytest.mark.parametrize("xt,ht,ot", [(F32, BF16, BF16), (BF16, F32, E4M3)])
def test_norm_of_large_outputs(M, d, xt, ht, ot):
    print(f"[large norm] {M}x{d} {xt} {ht} {ot}", flush=True)
    x, r, w = normal(1, (M, d), xt), normal(2, (M, d), ht, 2.0), normal(3, (d,), BF16)
    assert M * d * (2 if ht == BF16 else 4) + M * d * (2 if ot == BF16 else 1) >= 32 << 20
    h, check = guarded(M, d, ht)
    got = tw.add_rmsnorm(x, w, 1e-6, residual=r, out_dtype=ot, h=h)
    check()
    part = M // 7 + 1  # calls that store as small ones do
    for i in range(0, M, part):
        few = tw.add_rmsnorm(x[i:i + part], w, 1e-6, residual=r[i:i + part], out_dtype=ot)
        assert torch.equal(few.h, got.h[i:i + part]) and torch.equal(few.rstd, got.rstd[i:i + part])
        assert torch.equal(few.n.view(torch.uint8), got.n[i:i + part].view(torch.uint8))
    rows = [0, 1, M // 2, M - 1]
    s = O.dropout(host(x)[rows], 0.1, SEED, OFFSET, host(r)[rows], O.keep_mask(M, d, 0.1, SEED, OFFSET, rows))
    h2 = tw.add_rmsnorm(x, w, 1e-6, residual=r, p=0.1, seed=SEED, offset=OFFSET).h
    close(host(h2)[rows], s, half_step(ht, s) * (1 + 2**-8) + 3 * U * (2 * np.abs(host(x)[rows]) + np.abs(host(r)[rows])), "h")
    assert torch.equal(h2, tw.dropout(x, 0.1, SEED, OFFSET, residual=r))


@pytest.mark.parametrize("M,d", LARGE)
@pytest.mark.parametrize("gt,ht,xt", [(F32, BF16, F32), (BF16, F32, BF16)])
def test_norm_backward_of_large_outputs(M, d, gt, ht, xt):
    print(f"[large norm backward] {M}x{d} {gt} {ht} {xt}", flush=True)
    dn, h, dh, w = normal(1, (M, d), gt), normal(2, (M, d), ht, 2.0), normal(3, (M, d), ht), normal(4, (d,), BF16)
    rstd = tw.add_rmsnorm(h, w, 1e-6).rstd
    dres, dx, dw = tw.add_rmsnorm_backward(dn, h, w, rstd, dh=dh, dx_dtype=xt)
    part = M // 7 + 1
    for i in range(0, M, part):
        at = slice(i, i + part)
        few = tw.add_rmsnorm_backward(dn[at], h[at], w, rstd[at], dh=dh[at], dx_dtype=xt)
        assert torch.equal(few[0], dres[at]) and torch.equal(few[1], dx[at])
    terms = dn.double() * h.double() * rstd.double()[:, None]
    close(host(dw), host(terms.sum(dim=0)), (M / 512 + 64) * U * host(terms.abs().sum(dim=0)), "dweight")
    rows = [0, 1, M // 2, M - 1]
    dn_, h_, w_, r_ = host(dn)[rows], host(h)[rows], host(w), host(rstd)[rows]
    want, _ = O.rmsnorm_backward(dn_, h_, w_, r_)
    g, xh = np.abs(dn_ * w_), np.abs(h_) * r_[:, None]
    mag = r_[:, None] * (g + xh * (g * xh).mean(axis=1)[:, None]) + np.abs(host(dh)[rows])
    want = want + host(dh)[rows]
    close(host(dres)[rows], want, half_step(ht, want) * (1 + 2**-8) + SUM * mag, "dres")
    drop = tw.add_rmsnorm_backward(dn, h, w, rstd, dh=dh, dx_dtype=xt, p=0.2, seed=SEED, offset=OFFSET)
    assert torch.equal(drop[0], dres) and torch.equal(drop[2], dw)
    wx = O.dropout(want, 0.2, SEED, OFFSET, keep=O.keep_mask(M, d, 0.2, SEED, OFFSET, rows))
    close(host(drop[1])[rows], wx, half_step(xt, wx) * (1 + 2**-8) + 2 * SUM * mag, "dx")


@pytest.mark.parametrize("M,d", LARGE)
@pytest.mark.parametrize("xt,yt", [(F32, BF16), (BF16, F32), (BF16, BF16)])
def test_dropout_of_large_outputs(M, d, xt, yt):
    print(f"[large dropout] {M}x{d} {xt} {yt}", flush=True)
    x, r = normal(1, (M, d), xt), normal(2, (M, d), yt)
    out, check = guarded(M, d, yt)
    y = tw.dropout(x, 0.3, SEED, OFFSET, residual=r, out=out)
    check()
    part = M // 7  # the mask is one of rows from 0 on
    assert torch.equal(tw.dropout(x[:part], 0.3, SEED, OFFSET, residual=r[:part]), y[:part])
    kept = tw.dropout(torch.ones_like(x), 0.3, SEED, OFFSET, out_dtype=F32)
    t = O.keep_threshold(0.3)
    assert ((kept == 0) | (kept == float(np.float32(65536.0 / (65536 - t))))).all()
    close(host(y), host(r.double() + x.double() * kept.double()),
          half_step(yt, host(y)) * (1 + 2**-7) + 3 * U * (host(r.abs()) + 2 * host(x.abs())), "y")
    rows = [0, M // 2, M - 1]
    assert np.array_equal(host(kept)[rows] != 0, O.keep_mask(M, d, 0.3, SEED, OFFSET, rows))


# ------------------------------------------------------------------ offsets past 32 bits
def test_long_norm_and_dropout():
    M, d = (1 << 18) + 1, 8201
    room(24)
    print(f"[large] norm backward and dropout of {M}x{d}", flush=True)
    rows = [0, 1, M // 2, M - 2, M - 1]
    h, dn, w = normal(1, (M, d), BF16), normal(2, (M, d), BF16), normal(3, (d,), BF16)
    r = tw.add_rmsnorm(h, w, 1e-6)
    n, rstd = O.rmsnorm(host(h[rows]), host(w), 1e-6)
    close(host(r.rstd[rows]), rstd, SUM * rstd, "rstd")
    close(host(r.n[rows]), n, half_step(BF16, n) * (1 + 2**-8) + 2 * SUM * np.abs(n), "n")
    dres, _, dw = tw.add_rmsnorm_backward(dn, h, w, r.rstd)
    want, _ = O.rmsnorm_backward(host(dn[rows]), host(h[rows]), host(w), host(r.rstd[rows]))
    g, xh = np.abs(host(dn[rows]) * host(w)), np.abs(host(h[rows])) * rstd[:, None]
    mag = rstd[:, None] * (g + xh * (g * xh).mean(axis=1)[:, None])
    close(host(dres[rows]), want, half_step(BF16, want) * (1 + 2**-8) + SUM * mag, "dres")
    assert torch.isfinite(dw).all()
    y = tw.dropout(h, 0.4, SEED, OFFSET)
    want = O.dropout(host(h[rows]), 0.4, SEED, OFFSET, keep=O.keep_mask(M, d, 0.4, SEED, OFFSET, rows))
    close(host(y[rows]), want, half_step(BF16, want) * (1 + 2**-7), "y")


def codes_of(seed, N, K, group):
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.rand((N, -(-K // group)), generator=g, device=DEV).add_(0.5).mul_(K**-0.5 / 5).to(BF16)
    return tw.Q4(codes, scales, None, K, group)


def units_of(W, units):
    b = W.codes[units].cpu().numpy()
    q = np.stack((b & 15, b >> 4), axis=-1).reshape(len(units), -1)[:, :W.K]
    return O.q4_dequantize(q, host(W.scales[units]), None, W.group)


@pytest.mark.parametrize("M", [3, 40])
def test_long_weight(M):
    """4.3 GB of codes: few rows and many."""
    N, K = (1 << 20) + 5, 8200
    room(8)
    print(f"[large] product {M}x{N}x{K}", flush=True)
    W = codes_of(1, N, K, 64)
    units = [0, 1, N // 2, N - 2, N - 1]
    w = units_of(W, units)
    for xt in (BF16, F32):
        x = normal(2, (M, K), xt)
        want = host(x) @ w.T
        close(host(tw.q4_matmul(x, W)[:, units]), want, (K + 512) * U * (np.abs(host(x)) @ np.abs(w).T), "y")


@pytest.mark.parametrize("N,K,gib", [(40, 8200, 24), (1 << 15, 40, 36)])
def test_long_x_and_y(N, K, gib):
    """4.3 GB of x, as it is and as planes, and 2^33 elements of y."""
    M = 1 << 18
    room(gib)
    print(f"[large] product {M}x{N}x{K}", flush=True)
    W = codes_of(1, N, K, 32)
    rows, units = [0, 1, M // 2, M - 2, M - 1], [0, N // 2, N - 1]
    w = units_of(W, units)
    x = normal(2, (M, K), BF16)
    for xt in (BF16, E4M3) if N == 40 else (BF16,):
        xs = x.to(xt)
        sx = torch.ones(M, device=DEV) if xt == E4M3 else None
        y = tw.q4_matmul(xs, W, x_scale=sx)
        xr = host(xs[rows].float())
        close(host(y[rows][:, units]), xr @ w.T, (K + 512) * U * (np.abs(xr) @ np.abs(w).T), "y")


def test_long_weight_quantized():
    N, K, group = (1 << 19) + 3, 8201, 128
    room(20)
    print(f"[large] quantize {N}x{K}", flush=True)
    W = normal(1, (N, K), BF16)
    q = tw.q4_quantize(W, group)
    units = [0, 1, N // 2, N - 2, N - 1]
    codes, scales = O.q4_quantize(host(W[units]), group)
    assert np.array_equal(host(q.scales[units]), scales)
    got = q.codes[units].cpu().numpy()
    got[:, -1] &= 15  # what pads a row
    want = O.pack_codes(codes)
    want[:, -1] &= 15
    assert np.array_equal(got, want)
