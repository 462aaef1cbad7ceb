"""Layer norm and its backward where a value of the row passes fp32's range on the way to a result that does
not: rows of large equal values at widths that leave lanes without columns, and rows whose
values are further apart than the largest fp32.

Bounds as in test_gpu_layernorm.py."""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, OFFSET, SEED, SUM, U, close, half_step, host, rand  # noqa: E402

# lanes with all columns, none and some, rows a wave and a workgroup, one block a thread and two
WIDTHS = [24, 200, 256, 512, 520, 1000, 1001, 2048, 5000, 9000, 16384]


def check_backward(h, w, eps, dn, dh=None, p=0.0, xt=None):
    """The gradients that belong to the kernel's own mean and rstd, as test_add_layernorm_backward does."""
    f = tw.add_layernorm(h, w, None, eps)
    args = dict(dh=dh, p=p, seed=SEED, offset=OFFSET, dx_dtype=xt)
    dres, dx, dw, db = tw.add_layernorm_backward(dn, h, w, f.mean, f.rstd, **args)
    dn_, h_, w_, m_, r_ = host(dn), host(h), host(w), host(f.mean), host(f.rstd)
    assert np.isfinite(m_).all() and np.isfinite(r_).all()
    want, want_w, want_b = O.layernorm_backward(dn_, h_, w_, m_, r_)
    g, xh = np.abs(dn_ * w_), np.abs(h_ - m_[:, None]) * r_[:, None]
    mag = r_[:, None] * (g + g.mean(axis=1, keepdims=True) + xh * (g * xh).mean(axis=1, keepdims=True))
    if dh is not None:
        want, mag = want + host(dh), mag + np.abs(host(dh))
    close(dres, want, half_step(h.dtype, want) * (1 + 2**-8) + SUM * mag, "dres")
    close(dw, want_w, 256 * U * np.abs(dn_ * xh).sum(axis=0), "dweight")
    close(db, want_b, 256 * U * np.abs(dn_).sum(axis=0), "dbias")
    keep = O.keep_mask(*h.shape, p, SEED, OFFSET, range(h.shape[0]))
    wx = O.dropout(want, p, SEED, OFFSET, keep=keep)
    close(dx, wx, half_step(dx.dtype, wx) * (1 + 2**-8) + 2 * SUM * mag, "dx")


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("ht,xt,p", [(F32, F32, 0.0), (BF16, F32, 0.25)])
def test_backward_of_rows_of_equal_values(d, ht, xt, p):
    """The deviations are zero, so dres = rstd (g - mean(g)) + dh and the row adds nothing to dweight, whatever its
    mean times rstd is (1 / sqrt(eps) for such rows)."""
    print(f"[layernorm equal rows] {d} {ht}", flush=True)
    rng = np.random.default_rng(d)
    values = (3e38, -3e38, 1.5e36, -4e33, 1e20, 0.0, 0.37)
    h = torch.stack([torch.full((d,), v, device=DEV) for v in values] + [rand(rng, (d,), F32)]).to(ht)
    dn, dh, w = rand(rng, h.shape, F32), rand(rng, h.shape, ht), rand(rng, (d,), BF16)
    for eps in (1e-5, 1e-12):
        check_backward(h, w, eps, dn, dh, p, xt)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("eps", [1e-5, 1e-12, 1e-30, 1e-35])
def test_rows_of_equal_values(d, eps):
    """out = bias, and its scale is the bias's, at any mean."""
    print(f"[layernorm equal rows, forward] {d} {eps}", flush=True)
    rng = np.random.default_rng(d)
    x = torch.stack([torch.full((d,), v, device=DEV) for v in (3e38, 1.5e36, -2e34, 1e30, -1e25, 1e10, 0.0)])
    w, b = rand(rng, (d,), F32), rand(rng, (d,), F32)
    for ot in (BF16, E4M3):
        got = tw.add_layernorm(x, w, b, eps, out_dtype=ot)
        assert torch.equal(got.mean, x[:, 0])
        want = np.broadcast_to(host(b), x.shape)
        if ot == BF16:
            close(got.n, want, half_step(BF16, want), "n")
            continue
        scale = np.full(len(x), np.abs(host(b)).max() / 448)
        close(got.scale, scale, 2 * U * scale, "scale")
        q = want / scale[:, None]
        close(got.n, q, half_step(E4M3, q) * (1 + 2**-6) + 4 * U * np.abs(q), "n")


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("ht", [F32, BF16])
def test_backward_of_rows_wider_than_the_range(d, ht):
    """A few values of one sign among many of the other: a deviation from the mean passes the largest fp32, its
    product with rstd is about sqrt(d). (rstd lies under 2^-126 there, where its steps are 2^-149: what is compared
    are the gradients that belong to the rstd that the forward left.)"""
    print(f"[layernorm wide rows] {d} {ht}", flush=True)
    rng = np.random.default_rng(d)
    h = torch.full((4, d), -3.3e38, device=DEV)
    h[0, d // 2], h[1, 0], h[1, d - 1] = 3.3e38, 3.3e38, 3.0e38
    h[2] = -h[1]
    h[3] = rand(rng, (d,), F32)
    h = h.to(ht)
    check_backward(h, rand(rng, (d,), BF16), 1e-5, rand(rng, h.shape, F32), rand(rng, h.shape, ht))
