"""Low-rank adapters on the GPU, through the binding, against the fp64 oracle.

Error bounds, u = 2^-24: products of bf16 are exact, fp32 rows and t enter as three bf16
parts that add up to them (2^-24 of them at most is lost). t is a sum of K products (times 3 parts), split over
workgroups and waves: under (K + 128) u sum|x A| (32 products a matrix instruction taken as 32
additions); y one of R products: (3 R + 64) u factor sum|t B| and t's error through |B|; the factor, its
product and the sum with the base 4 u of their magnitudes; bf16 2^-8 of the value on top."""

from __future__ import annotations

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, U, close, half_step, host, q4_x, rand  # noqa: E402


def adapters(rng, n, N, K, R, scaling=True):
    return tw.Adapters(rand(rng, (n, R, K), BF16, K**-0.5), rand(rng, (n, N, R), BF16),
                       rand(rng, (n,), F32).abs() + 0.5 if scaling else None)


def check(y, x, index, a, base):
    A, B = host(a.A), host(a.B)
    n, R, K = A.shape
    f = np.ones(n) if a.scaling is None else host(a.scaling)
    index, b = index.cpu().numpy(), host(base)
    want = O.lora(x, index, A, B, f, b)
    bound = np.zeros_like(want)
    for m, i in enumerate(index):
        if 0 <= i < n:
            t, e_t = np.abs(A[i] @ x[m]), (K + 128) * U * (np.abs(A[i]) @ np.abs(x[m]))
            t = t + e_t
            part = f[i] * (np.abs(B[i]) @ ((3 * R + 64) * U * t + e_t))
            bound[m] = part + 4 * U * (f[i] * (np.abs(B[i]) @ t) + np.abs(b[m]))
    none = (index < 0) | (index >= n)
    assert torch.equal(y[torch.from_numpy(none).to(DEV)], base[torch.from_numpy(none).to(DEV)])
    close(y, want, half_step(base.dtype, want) * (1 + 2**-8) + bound, "y")


# M, N, K, R, adapters
SIZES = [(1, 1, 1, 1, 1), (1, 64, 2048, 16, 4), (2, 33, 40, 3, 2), (5, 100, 129, 8, 3), (16, 65, 515, 7, 5),
         (17, 257, 300, 16, 17), (33, 48, 1024, 17, 2), (64, 130, 2560, 32, 48), (65, 31, 640, 33, 9), (100, 72, 96, 64, 200),
         (40, 24, 383, 65, 6), (20, 40, 256, 128, 3), (18, 520, 200, 256, 2), (300, 129, 4100, 24, 11), (257, 16, 64, 200, 40),
         (3, 2051, 8192, 16, 2), (1100, 96, 512, 16, 7),
         # multiples of 64 all over: one part and unit of N and many, each number of r, waves without steps of K, long K
         (1, 64, 64, 8, 1), (2, 128, 64, 16, 2), (16, 192, 128, 24, 5), (17, 8192, 192, 32, 3), (64, 256, 8192, 16, 48),
         (33, 64, 5120, 32, 8), (40, 320, 320, 40, 30), (70, 704, 2048, 48, 3), (90, 128, 4160, 56, 90), (300, 1024, 256, 64, 5),
         (256, 64, 128, 8, 300), (257, 2560, 64, 8, 4), (600, 128, 64, 16, 1000), (2000, 64, 64, 32, 2)]


@pytest.mark.parametrize("M,N,K,R,n", SIZES)
@pytest.mark.parametrize("xt,yt", [(BF16, F32), (F32, F32), (E4M3, BF16), (F32, BF16), (BF16, BF16)])
def test_lora_add(M, N, K, R, n, xt, yt):
    print(f"[lora] {M}x{N}x{K} r{R} n{n} {xt} {yt}", flush=True)
    rng = np.random.default_rng(M * 3 + N + K)
    x, sx, xr = q4_x(rng, M, K, xt)
    a = adapters(rng, n, N, K, R)
    # every adapter, none (-1), and numbers past the last
    index = torch.from_numpy(rng.integers(-1, n + 1, M).astype(np.int32)).to(DEV)
    if M == 1:
        index.fill_(n - 1)
    base = rand(rng, (M, N), yt)
    y = tw.lora_add(x, a, index, base, x_scale=sx)
    check(y, xr, index, a, base)
    again = base.clone()
    assert tw.lora_add(x, a, index, again, x_scale=sx, y=again) is again
    assert torch.equal(y, again)


@pytest.mark.parametrize("M", [1, 15, 16, 17, 40, 256, 257, 700])
@pytest.mark.parametrize("N,K", [(96, 520), (128, 512)])
def test_orders_of_requests(M, N, K):
    """One adapter for all, one each, runs, alternating, none: a row's result depends on its own
    adapter alone, so all agree bit for bit with a call of that row's adapter for every row."""
    print(f"[lora orders] {M} {N} {K}", flush=True)
    rng = np.random.default_rng(M)
    R, n = 16, 20
    x, base = rand(rng, (M, K), F32), rand(rng, (M, N), F32)
    a = adapters(rng, n, N, K, R, scaling=False)
    whole = [tw.lora_add(x, a, torch.full((M,), i, dtype=torch.int32, device=DEV), base) for i in range(n)]
    check(whole[3], host(x), torch.full((M,), 3, dtype=torch.int32), a, base)
    rows = np.arange(M)
    for order in (rows % n, rows // 7 % n, rows % 2 * 5, rng.integers(0, n, M), (rows // 16) % n, np.full(M, n - 1)):
        index = torch.from_numpy(order.astype(np.int32)).to(DEV)
        y = tw.lora_add(x, a, index, base)
        want = torch.stack(whole)[index.long(), torch.arange(M, device=DEV)]
        assert torch.equal(y, want)
    for none in (-1, n, -(1 << 31), (1 << 31) - 1):
        y = tw.lora_add(x, a, torch.full((M,), none, dtype=torch.int32, device=DEV), base)
        assert torch.equal(y, base) and y.data_ptr() != base.data_ptr()


def test_forms():
    """No adapters at all, ranks padded with zeros, odd addresses, guarded outputs."""
    rng = np.random.default_rng(4)
    x, base = rand(rng, (20, 100), BF16), rand(rng, (20, 50), F32)
    index = torch.zeros(20, dtype=torch.int32, device=DEV)
    none = tw.Adapters(torch.empty(0, 4, 100, dtype=BF16, device=DEV), torch.empty(0, 50, 4, dtype=BF16, device=DEV))
    assert torch.equal(tw.lora_add(x, none, index, base), base)
    a = adapters(rng, 2, 50, 100, 5)
    wide = tw.Adapters(torch.zeros(2, 16, 100, dtype=BF16, device=DEV), torch.zeros(2, 50, 16, dtype=BF16, device=DEV), a.scaling)
    wide.A[:, :5], wide.B[:, :, :5] = a.A, a.B
    y = tw.lora_add(x, a, index, base)
    assert torch.equal(tw.lora_add(x, wide, index, base), y)

    def odd(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:].copy_(t.flatten())
        return flat[1:].view(t.shape)

    b = tw.Adapters(odd(a.A), odd(a.B), odd(a.scaling))
    assert torch.equal(tw.lora_add(odd(x), b, odd(index), odd(base)), y)
    for N in (50, 63, 256, 257):
        a = adapters(rng, 2, N, 100, 5)
        for t in (F32, BF16):
            big = torch.full((20 * N + 64,), 7.0, device=DEV).to(t)
            inner = big[32:32 + 20 * N].view(20, N)
            tw.lora_add(x, a, index, rand(rng, (20, N), t), y=inner)
            assert (big[:32] == 7).all() and (big[-32:] == 7).all() and not (inner == 7).all()
    empty = torch.empty(0, 100, dtype=BF16, device=DEV)
    assert tw.lora_add(empty, a, index[:0], torch.empty(0, 257, device=DEV)).shape == (0, 257)


def test_values_that_are_not_finite_stay_in_their_rows():
    rng = np.random.default_rng(5)
    M, N, K, R, n = 40, 70, 200, 12, 4
    for xt in (BF16, F32):
        x, base = rand(rng, (M, K), xt), rand(rng, (M, N), F32)
        a = adapters(rng, n, N, K, R)
        index = torch.from_numpy(rng.integers(0, n, M).astype(np.int32)).to(DEV)
        want = tw.lora_add(x, a, index, base)
        x2, base2 = x.clone(), base.clone()
        x2[3, 5], x2[17, 199], x2[18, 0], base2[30, 2] = float("nan"), float("inf"), float("-inf"), float("nan")
        y = tw.lora_add(x2, a, index, base2)
        bad = torch.zeros(M, dtype=torch.bool, device=DEV)
        bad[[3, 17, 18]] = True
        assert not torch.isfinite(y[bad]).any()
        assert torch.isnan(y[30, 2])
        y[30, 2] = want[30, 2]
        assert torch.equal(y[~bad], want[~bad])
        # an adapter that is not finite spoils its own rows only
        a2 = tw.Adapters(a.A.clone(), a.B.clone(), a.scaling)
        a2.A[1, 2, 3], a2.B[2, 5, 6] = float("nan"), float("inf")
        y = tw.lora_add(x, a2, index, base)
        assert not torch.isfinite(y[index == 1]).any() and not torch.isfinite(y[index == 2][:, 5]).any()
        other = (index == 0) | (index == 3)
        assert torch.equal(y[other], want[other])
        keep = [c for c in range(N) if c != 5]
        assert torch.equal(y[index == 2][:, keep], want[index == 2][:, keep])


@pytest.mark.parametrize("start", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K,R", [(1, 1, 1, 1), (3, 2, 5, 1), (17, 33, 71, 3), (20, 41, 130, 7), (18, 72, 263, 9), (5, 50, 96, 21),
                                     (16, 31, 33, 70), (2, 65, 1032, 130)])
def test_odd_starts_between_values_that_are_not_finite(M, N, K, R, start):
    """Operands that begin at any element, with infinities and NaN before and behind, in the rows of x that have no
    adapter and in the adapters that no row names; outputs between values that stay."""
    rng = np.random.default_rng(M + N + K + R)
    index = torch.from_numpy(rng.integers(1, 3, M).astype(np.int32)).to(DEV) * 2 - 1  # 1 and 3 of 0..3, 3 the last
    if M > 2:
        index[1] = -1

    def between(t, around):
        flat = torch.full((t.numel() + 16,), around, dtype=F32, device=DEV).to(t.dtype)
        inner = flat[start:start + t.numel()].view(t.shape)
        inner.copy_(t)
        return inner, flat

    for xt, yt in ((BF16, F32), (F32, BF16), (E4M3, BF16)):
        print(f"[lora] odd start {start} {M}x{N}x{K} r{R} {xt} {yt}", flush=True)
        x, sx, xr = q4_x(rng, M, K, xt)
        x = x.clone()
        if M > 2:
            x[1] = torch.full((K,), float("nan"), device=DEV).to(xt)
        a = adapters(rng, 4, N, K, R)
        a.A[0], a.A[2], a.B[0], a.B[2] = float("nan"), float("inf"), float("inf"), float("nan")
        base = rand(rng, (M, N), yt)
        want = tw.lora_add(x, a, index, base, x_scale=sx)
        rows = torch.arange(M, device=DEV) != 1 if M > 2 else torch.ones(M, dtype=torch.bool, device=DEV)
        at = rows.cpu().numpy()
        used = tw.Adapters(a.A[[1, 3]].contiguous(), a.B[[1, 3]].contiguous(), a.scaling[[1, 3]].contiguous())
        check(want[rows], xr[at], (index[rows] - 1) // 2, used, base[rows])
        shifted = tw.Adapters(between(a.A, float("inf"))[0], between(a.B, float("nan"))[0], a.scaling)
        out, flat = between(torch.zeros_like(base), 7.0)
        y = tw.lora_add(between(x, float("nan"))[0], shifted, index, between(base, float("nan"))[0], x_scale=sx, y=out)
        assert torch.equal(y, want)
        assert (flat[:start] == 7).all() and (flat[start + M * N:] == 7).all()


def test_small_and_large_values():
    """fp32 rows over the range: three bf16 parts hold all of a value down to 2^-110 (2^-133 is bf16's least
    step), t is then 2^-133 off a product at most."""
    rng = np.random.default_rng(6)
    M, N, K, R = 12, 40, 64, 8
    base = torch.zeros(M, N, device=DEV)
    a = adapters(rng, 1, N, K, R, scaling=False)
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    for e in (-100, -60, 0, 60, 110):
        x = rand(rng, (M, K), F32).clamp(-4, 4) * 2.0**e
        check(tw.lora_add(x, a, index, base), host(x), index, a, base)


def test_large_offsets():
    """Adapters past 2^31 elements, and y past 2^32."""
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < 60 << 30:
        pytest.skip("needs 60 GiB of device memory")
    print("[lora] large offsets", flush=True)
    rng = np.random.default_rng(7)
    n, R, K, N = 3, 256, 1 << 22, 24
    A = torch.zeros(n, R, K, dtype=BF16, device=DEV)
    A[2, 255, K - 1], A[2, 0, 5] = 2.0, 3.0
    a = tw.Adapters(A, rand(rng, (n, N, R), BF16))
    x, base = torch.zeros(2, K, dtype=BF16, device=DEV), torch.zeros(2, N, device=DEV)
    x[1, K - 1], x[1, 5] = 1.5, -1.0
    y = tw.lora_add(x, a, torch.tensor([0, 2], dtype=torch.int32, device=DEV), base)
    want = 3.0 * host(a.B)[2, :, 255] - 3.0 * host(a.B)[2, :, 0]
    assert (y[0] == 0).all()
    close(host(y)[1], want, 8 * U * 3 * (np.abs(host(a.B)[2, :, 255]) + np.abs(host(a.B)[2, :, 0])), "y")
    del A, a
    torch.cuda.empty_cache()
    M, N, K, R = 1 << 14, (1 << 18) + 8, 8, 1
    x = torch.ones(M, K, dtype=BF16, device=DEV)
    a = tw.Adapters(torch.ones(1, R, K, dtype=BF16, device=DEV), torch.ones(1, N, R, dtype=BF16, device=DEV))
    base = torch.ones(1, 1, dtype=BF16, device=DEV).expand(M, N).contiguous()
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    index[M // 2] = -1
    tw.lora_add(x, a, index, base, y=base)
    for i in range(0, M, 1 << 10):
        part = base[i:i + (1 << 10)]
        rows = torch.full((part.shape[0], 1), 9.0, device=DEV, dtype=BF16)
        if i <= M // 2 < i + (1 << 10):
            rows[M // 2 - i] = 1.0
        assert bool((part == rows).all()), i
    del base
    torch.cuda.empty_cache()


def test_beside_the_shared_projection():
    """q4_matmul's output as the base, in place, as a program calls them; captured, replayed with eager work between, and on two
    streams at once."""
    rng = np.random.default_rng(8)
    M, N, K, R, n = 24, 320, 512, 16, 6
    W = tw.q4_quantize(rand(rng, (N, K), BF16, K**-0.5))
    a = adapters(rng, n, N, K, R)
    x = rand(rng, (M, K), BF16)
    index = torch.from_numpy(rng.integers(-1, n, M).astype(np.int32)).to(DEV)

    def project():
        y = tw.q4_matmul(x, W)
        return tw.lora_add(x, a, index, y, y=y)

    check(project(), host(x), index, a, tw.q4_matmul(x, W))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = project()
    for k in range(4):
        x.copy_(rand(rng, (M, K), BF16))
        index.copy_(torch.from_numpy(rng.integers(-1, n, M).astype(np.int32)))
        want = project()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
    want = project()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(project())
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_refusals():
    rng = np.random.default_rng(9)
    x, base = rand(rng, (4, 32), BF16), rand(rng, (4, 16), F32)
    a = adapters(rng, 2, 16, 32, 3)
    index = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (lambda: tw.lora_add(x, a, index[:3], base), lambda: tw.lora_add(x, a, index, base[:, :15]),
                lambda: tw.lora_add(x[:, :31].contiguous(), a, index, base),
                lambda: tw.lora_add(x, tw.Adapters(a.A, a.B[:1], a.scaling), index, base),
                lambda: tw.lora_add(x, tw.Adapters(a.A[0], a.B, a.scaling), index, base),
                lambda: tw.lora_add(x, tw.Adapters(a.A, a.B, a.scaling[:1]), index, base),
                lambda: tw.lora_add(x, a, index, base, x_scale=torch.ones(4, device=DEV)),
                lambda: tw.lora_add(x.to(E4M3), a, index, base), lambda: tw.lora_add(x.cpu(), a, index, base),
                lambda: tw.lora_add(x, a, index.cpu(), base)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tw.lora_add(x, a, index.long(), base), lambda: tw.lora_add(x, a, index, base.half()),
                lambda: tw.lora_add(x, a, index, base, y=base.bfloat16()),
                lambda: tw.lora_add(x, tw.Adapters(a.A.float(), a.B), index, base)):
        with pytest.raises(TypeError):
            bad()
    big = tw.Adapters(torch.zeros(1, 257, 32, dtype=BF16, device=DEV), torch.zeros(1, 16, 257, dtype=BF16, device=DEV))
    with pytest.raises(tw.TwellError):
        tw.lora_add(x, big, index, base)
