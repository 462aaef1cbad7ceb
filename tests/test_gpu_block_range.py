"""The residual norm over fp32's range: rows whose squares pass it in either
direction, against the fp64 oracle. Bounds: rstd 2^-17 (the sums) and 2^-149 (the
step of numbers below 2^-126, which the rstd of the largest rows is), out twice that
and its own rounding."""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, SUM, close, half_step, host, rand  # noqa: E402

POWERS = (-120, -100, -75, -65, -50, 0, 40, 58, 60, 62, 64, 100, 124)


@pytest.mark.parametrize("d", [24, 512, 1000, 5000, 12001])
@pytest.mark.parametrize("ht", [F32, BF16])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-35])
def test_norm_of_small_and_large_rows(d, ht, eps):
    print(f"[norm range] d={d} {ht} eps={eps}", flush=True)
    rng = np.random.default_rng(d)
    x = torch.stack([rand(rng, (d,), F32).clamp(-7, 7) * 2.0**e for e in POWERS]).to(ht)
    w = rand(rng, (d,), BF16)
    s, wr = host(x), host(w)
    n, rstd = O.rmsnorm(s, wr, float(np.float32(eps)))
    for ot in (BF16, E4M3):
        got = tw.add_rmsnorm(x, w, eps, residual=torch.zeros_like(x), out_dtype=ot)
        assert torch.equal(got.h, x)
        close(got.rstd, rstd, SUM * rstd + 2.0**-149, "rstd")
        slack = 2 * SUM * np.abs(n) + np.abs(s * wr) * 2.0**-149
        if ot == BF16:
            close(got.n, n, half_step(BF16, n) * (1 + 2**-8) + slack, "n")
            continue
        scale = np.maximum(np.abs(n).max(axis=1), 2.0**-100) / 448
        err = slack.max(axis=1) / 448
        close(got.scale, scale, 4 * SUM * scale + err, "scale")
        q = n / scale[:, None]
        close(got.n, q, half_step(E4M3, q) * (1 + 2**-7) + slack / scale[:, None] + (8 * SUM + err / scale)[:, None] * np.abs(q),
              "n")


def test_rows_of_infinities_and_lowest_values():
    for d in (40, 2048, 9000):
        x = torch.randn(5, d, device=DEV)
        x[1, 3] = float("inf")
        x[2] = torch.finfo(BF16).min
        x[3, d - 1] = torch.finfo(F32).min
        x[4] = 0
        got = tw.add_rmsnorm(x, torch.ones(d, device=DEV), 1e-6)
        n = got.n.float()
        assert got.rstd[1] == 0 and torch.isnan(n[1, 3])
        assert (n[2] == -1).all()
        assert n[3, d - 1] == torch.tensor(-(d**0.5)).bfloat16()
        assert (n[3, : d - 1].abs() < 1e-35).all() and (n[4] == 0).all()
