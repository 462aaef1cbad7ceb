"""Low-rank adapters at widths that are whole blocks (K and N multiples of 64, R of 8 up to 64), whose operands go
through LDS, beside the same at other widths: values that are not finite and memory around the operands,
the ends of fp32's range, and offsets at the ends of what is addressed.

Bounds as in test_gpu_lora.py."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU only to be deselected by -m
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_ffn_gate_amd as tw  # noqa: E402
from test_gpu_block import BF16, DEV, E4M3, F32, U, close, host, q4_x, rand  # noqa: E402
from test_gpu_lora import adapters, check  # noqa: E402

# M, N, K, R: 16, 32 and 64 r; some waves without a step, a long K in 8 and in 16 waves; one item and several
BLOCKS = [(5, 128, 256, 8), (16, 64, 64, 16), (40, 192, 320, 24), (300, 128, 512, 40), (20, 64, 4160, 16), (33, 256, 8192, 32),
          (257, 64, 4096, 64), (70, 1024, 192, 56)]


def between(t, around, start):
    """The same values between others."""
    flat = torch.full((t.numel() + 16,), around, dtype=F32, device=DEV).to(t.dtype)
    inner = flat[start:start + t.numel()].view(t.shape)
    inner.copy_(t)
    return inner, flat


@pytest.mark.parametrize("M,N,K,R", BLOCKS)
@pytest.mark.parametrize("xt,yt", [(BF16, F32), (F32, F32), (E4M3, F32), (BF16, BF16), (F32, BF16)])
def test_values_that_are_not_finite_stay_in_their_rows(M, N, K, R, xt, yt):
    """Rows of x with an adapter and without one, adapters that no row names and one that some rows do; operands
    between values that are not finite, outputs between values that stay."""
    print(f"[lora blocks] {M}x{N}x{K} r{R} {xt} {yt}", flush=True)
    rng = np.random.default_rng(M + N + K + R)
    x, sx, xr = q4_x(rng, M, K, xt)
    a = adapters(rng, 6, N, K, R)
    a.A[0], a.A[2], a.B[0], a.B[2] = float("nan"), float("inf"), float("inf"), float("nan")
    base = rand(rng, (M, N), yt)
    named = np.array([1, 3, 4, 5])  # the last one's memory ends the tensors
    index = named[rng.integers(0, 4, M)].astype(np.int32)
    index[1], index[M // 2] = -1, 5
    none = index == -1
    index = torch.from_numpy(index).to(DEV)
    want = tw.lora_add(x, a, index, base, x_scale=sx)
    used = tw.Adapters(a.A[named].contiguous(), a.B[named].contiguous(), a.scaling[named].contiguous())
    check(want, xr, torch.from_numpy(np.where(none, -1, np.searchsorted(named, index.cpu().numpy()))), used, base)

    # memory around: the aligned place that whole blocks need, and places one to three elements past one
    for start in (0, 8, 1, 2, 3):
        y, flat = between(torch.zeros_like(base), 7.0, start)
        if start in (0, 8):
            shifted = tw.Adapters(between(a.A, float("inf"), start)[0], between(a.B, float("nan"), start)[0], a.scaling)
            z = between(x, float("nan"), 0 if xt == E4M3 else start)[0]
        else:  # base and y alone
            shifted, z = a, x
        tw.lora_add(z, shifted, index, between(base, float("nan"), start)[0], x_scale=sx, y=y)
        assert torch.equal(y, want), start
        assert (flat[:start] == 7).all() and (flat[start + M * N:] == 7).all(), start
        over, flat = between(base, 7.0, start)
        assert torch.equal(tw.lora_add(z, shifted, index, over, x_scale=sx, y=over), want), start
        assert (flat[:start] == 7).all() and (flat[start + M * N:] == 7).all(), start

    # rows: one without an adapter, three with one
    x2, bad = x.clone(), torch.zeros(M, dtype=torch.bool, device=DEV)
    rows = sorted({0, M // 2, M - 1})
    raw = x2.view(torch.uint8) if xt == E4M3 else x2
    for r, c in zip(rows, (0, K // 2, K - 1)):
        raw[r, c] = 0x7F if xt == E4M3 else float("nan") if r else float("inf")
    raw[1] = 0x7F if xt == E4M3 else float("nan")
    bad[rows] = True
    y = tw.lora_add(x2, a, index, base, x_scale=sx)
    assert torch.equal(y[~bad], want[~bad]) and not torch.isfinite(y[bad]).any()

    # an adapter: a row of A spoils its rows, a value of B one column of them
    a2 = tw.Adapters(a.A.clone(), a.B.clone(), a.scaling)
    a2.A[4, R - 1, K - 1], a2.B[3, 5, R - 1], a2.B[3, N - 1, 0] = float("nan"), float("inf"), float("nan")
    y = tw.lora_add(x, a2, index, base, x_scale=sx)
    assert not torch.isfinite(y[index == 4]).any()
    three = index == 3
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[[5, N - 1]] = False
    assert not torch.isfinite(y[three][:, ~keep]).any() and torch.equal(y[three][:, keep], want[three][:, keep])
    other = (index != 3) & (index != 4)
    assert torch.equal(y[other], want[other])


@pytest.mark.parametrize("M,N,K,R", [(5, 128, 256, 8), (40, 64, 320, 24), (33, 128, 4160, 16), (20, 64, 64, 64)])
def test_small_and_large_values(M, N, K, R):
    """fp32 rows over the range, from which up to 512 values are cut into parts at a time: as at other widths."""
    print(f"[lora blocks range] {M}x{N}x{K} r{R}", flush=True)
    rng = np.random.default_rng(K)
    a = adapters(rng, 3, N, K, R, scaling=False)
    index = torch.from_numpy(rng.integers(0, 3, M).astype(np.int32)).to(DEV)
    base = torch.zeros(M, N, device=DEV)
    for e in (-100, -60, 0, 60, 110):
        x = rand(rng, (M, K), F32).clamp(-4, 4) * 2.0**e
        check(tw.lora_add(x, a, index, base), host(x), index, a, base)
    # rows of different sizes beside each other
    x = rand(rng, (M, K), F32).clamp(-4, 4) * torch.from_numpy(2.0 ** rng.integers(-100, 100, M)).to(DEV, F32)[:, None]
    check(tw.lora_add(x, a, index, base), host(x), index, a, base)


@pytest.mark.parametrize("M,N,K,R", [(5, 128, 256, 8), (18, 64, 128, 48), (6, 70, 200, 12), (17, 33, 71, 3), (5, 64, 128, 72)])
def test_values_next_to_the_largest(M, N, K, R):
    """fp32 values of x, and of t, that no bf16 of 8 bits rounded to nearest holds: the largest bf16 is 2^-9 below the
    largest fp32."""
    print(f"[lora blocks largest] {M}x{N}x{K} r{R}", flush=True)
    rng = np.random.default_rng(R)
    largest = torch.finfo(F32).max
    a = adapters(rng, 2, N, K, R, scaling=False)
    a.A[0] *= 2.0**-20  # of many values
    a.B[0].clamp_(-2, 2)
    a.A[1], a.B[1] = 0, a.B[1].clamp(-2, 2) * 2.0**-10
    a.A[1, :, K // 3] = 1  # t is the largest itself
    x = rand(rng, (M, K), F32)
    x[0, 0], x[1, K - 1], x[2, K // 3], x[3, K // 3], x[4, K // 3] = largest, -largest, largest, -largest, largest * (1 - 2.0**-10)
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    index[2:5] = 1
    base = rand(rng, (M, N), F32)
    y = tw.lora_add(x, a, index, base)
    assert torch.isfinite(y).all()
    check(y, host(x), index, a, base)


def test_long_rows_of_fp32():
    """A block of 256 rows of 2^22 fp32 values: 32-bit offsets in it end 2 KB below 2^32."""
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < 30 << 30:
        pytest.skip("needs 30 GiB of device memory")
    print("[lora blocks] long rows", flush=True)
    rng = np.random.default_rng(7)
    M, N, K, R, n = 256, 64, 1 << 22, 8, 2
    a = tw.Adapters(torch.zeros(n, R, K, dtype=BF16, device=DEV), rand(rng, (n, N, R), BF16))
    a.A[0, 0, 0], a.A[0, R - 1, K - 1], a.A[1, 3, K - 1], a.A[1, R - 1, K // 2 + 5] = 1.0, 2.0, 3.0, -1.0
    x = torch.zeros(M, K, device=DEV)
    x[:, 0], x[:, K - 1], x[:, K // 2 + 5] = (torch.arange(M, device=DEV) * i + 1.0 for i in (1, 2, 3))
    index = (torch.arange(M, device=DEV) % 3).to(torch.int32)  # 2: none
    y = tw.lora_add(x, a, index, torch.zeros(M, N, device=DEV))
    B, rows = host(a.B), np.arange(M)
    want, mag = np.zeros((M, N)), np.zeros((M, N))
    for i, terms in ((0, (((1, 0), 1.0), ((2, R - 1), 2.0))), (1, (((2, 3), 3.0), ((3, R - 1), -1.0)))):
        for (slope, r), f in terms:
            part = np.outer(f * (rows * slope + 1.0), B[i, :, r]) * (rows % 3 == i)[:, None]
            want, mag = want + part, mag + np.abs(part)
    close(y, want, 8 * U * mag, "y")  # t is exact, two products of three parts each are added
    del x, a
    torch.cuda.empty_cache()


def test_outputs_past_32_bits():
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < 60 << 30:
        pytest.skip("needs 60 GiB of device memory")
    print("[lora blocks] outputs past 32 bits", flush=True)
    M, N, K, R = 1 << 14, (1 << 18) + 64, 64, 8
    x = torch.ones(M, K, dtype=BF16, device=DEV)
    a = tw.Adapters(torch.ones(1, R, K, dtype=BF16, device=DEV), torch.ones(1, N, R, dtype=BF16, device=DEV))
    base = torch.ones(1, 1, dtype=BF16, device=DEV).expand(M, N).contiguous()
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    index[M // 2] = -1
    tw.lora_add(x, a, index, base, y=base)
    want = torch.tensor(1.0 + K * R, device=DEV).to(BF16)
    for i in range(0, M, 1 << 10):
        rows = want.expand(1 << 10, 1).clone()
        if i <= M // 2 < i + (1 << 10):
            rows[M // 2 - i] = 1.0
        assert bool((base[i:i + (1 << 10)] == rows).all()), i
    del base
    torch.cuda.empty_cache()


def test_widest_rows():
    """N = 2^22 with a block of 256 rows: offsets in it end at 2^32."""
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < 30 << 30:
        pytest.skip("needs 30 GiB of device memory")
    print("[lora blocks] widest rows", flush=True)
    M, N, K, R = 256, 1 << 22, 64, 8
    x = torch.ones(M, K, dtype=BF16, device=DEV)
    x[:, 0] = torch.arange(M, device=DEV).to(BF16)
    a = tw.Adapters(torch.zeros(1, R, K, dtype=BF16, device=DEV), torch.ones(1, N, R, dtype=BF16, device=DEV))
    a.A[0, 0, 0] = 1.0  # t[m, 0] = m, which bf16 holds up to 256
    a.B[0, N - 1, 0], a.B[0, 0, 0] = 2.0, 3.0
    y = torch.zeros(M, N, device=DEV)
    tw.lora_add(x, a, torch.zeros(M, dtype=torch.int32, device=DEV), y, y=y)
    rows = torch.arange(M, device=DEV, dtype=F32)
    assert torch.equal(y[:, N - 1], 2 * rows) and torch.equal(y[:, 0], 3 * rows)
    for i in range(0, M, 32):
        assert bool((y[i:i + 32, 1:N - 1] == rows[i:i + 32, None]).all()), i
    del y, a
    torch.cuda.empty_cache()


def test_refuses_y_in_part_of_its_operands():
    """Before anything is enqueued; views of one buffer that only touch are fine."""
    rng = np.random.default_rng(3)
    M, N, K, R = 4, 64, 128, 8
    buf = torch.zeros(4 * M * N, device=DEV)
    a = adapters(rng, 2, N, K, R)
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    base = buf[M * N:2 * M * N].view(M, N)
    base.copy_(rand(rng, (M, N), F32))
    x = buf[2 * M * N:2 * M * N + M * K].view(M, K)
    x.copy_(rand(rng, (M, K), F32))
    kept = buf.clone()
    for first in (1, M * N - 1, M * N + 1, 2 * M * N - 1, 2 * M * N, 2 * M * N + 7):
        with pytest.raises(tw.TwellError):
            tw.lora_add(x, a, index, base, y=buf[first:first + M * N].view(M, N))
    assert torch.equal(buf, kept)
    want = tw.lora_add(x, a, index, base)
    assert torch.equal(tw.lora_add(x, a, index, base, y=buf[:M * N].view(M, N)), want)
    assert torch.equal(tw.lora_add(x, a, index, base, y=base), want)
