"""Operators around the FFN at sizes of memory: rows past what one dimension of a
launch holds, outputs that are stored past the L2. Against the fp64 oracle, with the
bounds of tests/test_gpu_block.py's kind: 2^-8 of a bf16 value and 2^-4 of an e4m3
one (or 2^-10), fp32 sums 2^-17 of their magnitude."""

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
