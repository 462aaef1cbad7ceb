"""Forms of the norm's C entries that the binding does not make: outputs left out,
gradients written where they came from. Bit for bit against the full calls."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, OFFSET, SEED, rand  # noqa: E402

TYPE = {BF16: 0, F32: 1, E4M3: 2}
SIZES = [(7, 129), (300, 512), (40, 1003), (9, 2560), (3, 9001)]


def _p(t):
    return None if t is None else t.data_ptr()


def _backward(dn, dh, h, w, rstd, p, dres, dx, dx_type, dw):
    M, d = dn.shape
    ws = tw.Workspace(DEV)
    wp, wn = ws.get(tw.rmsnorm_workspace_bytes(M, d))
    st = tw.lib().twell_add_rmsnorm_backward(
        _p(dn), TYPE[dn.dtype], _p(dh), _p(h), TYPE[h.dtype], _p(w), TYPE[w.dtype], _p(rstd), M, d, p, SEED, OFFSET,
        _p(dres), _p(dx), TYPE[dx_type], _p(dw), wp, wn, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()  # the workspace is held until the call has run


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("gt,ht,xt", [(F32, BF16, BF16), (BF16, F32, BF16), (F32, F32, F32)])
def test_backward_outputs_left_out_or_in_place(M, d, p, gt, ht, xt):
    print(f"[norm forms] backward {M}x{d} p={p} {gt} {ht} {xt}", flush=True)
    rng = np.random.default_rng(M + d)
    dn, h, dh, w = rand(rng, (M, d), gt), rand(rng, (M, d), ht, 2.0), rand(rng, (M, d), ht), rand(rng, (d,), F32)
    rstd = tw.add_rmsnorm(h, w, 1e-5).rstd
    dres, dx, dw = tw.add_rmsnorm_backward(dn, h, w, rstd, dh=dh, p=p, seed=SEED, offset=OFFSET, dx_dtype=xt)
    for left_out in ("dres", "dx"):
        a, b, c = torch.empty_like(dres), torch.empty((M, d), dtype=xt, device=DEV), torch.empty_like(dw)
        _backward(dn, dh, h, w, rstd, p, None if left_out == "dres" else a, None if left_out == "dx" else b, xt, c)
        assert torch.equal(c, dw)
        assert torch.equal(b, dx) if left_out == "dres" else torch.equal(a, dres)
    a, b, c = dh.clone(), torch.empty((M, d), dtype=xt, device=DEV), torch.empty_like(dw)
    _backward(dn, a, h, w, rstd, p, a, b, xt, c)  # the gradient of h becomes that of residual
    assert torch.equal(a, dres) and torch.equal(b, dx) and torch.equal(c, dw)


@pytest.mark.parametrize("M,d", SIZES)
@pytest.mark.parametrize("ot", [BF16, E4M3])
def test_forward_outputs_left_out(M, d, ot):
    print(f"[norm forms] forward {M}x{d} {ot}", flush=True)
    rng = np.random.default_rng(M + d)
    x, r, w = rand(rng, (M, d), F32), rand(rng, (M, d), BF16), rand(rng, (d,), BF16)
    want = tw.add_rmsnorm(x, w, 1e-5, residual=r, p=0.3, seed=SEED, offset=OFFSET, out_dtype=ot)
    for h, rstd in ((None, True), (True, None), (None, None)):
        h = None if h is None else torch.empty_like(r)
        rstd = None if rstd is None else torch.empty(M, device=DEV)
        n = torch.empty((M, d), dtype=ot, device=DEV)
        scale = torch.empty(M, device=DEV) if ot == E4M3 else None
        st = tw.lib().twell_add_rmsnorm(_p(x), 1, _p(r), _p(w), 0, M, d, 1e-5, 0.3, SEED, OFFSET, _p(h), 0, _p(n),
                                        TYPE[ot], _p(scale), _p(rstd), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(n.view(torch.uint8), want.n.view(torch.uint8))
        assert h is None or torch.equal(h, want.h)
        assert rstd is None or torch.equal(rstd, want.rstd)
        assert scale is None or torch.equal(scale, want.scale)
