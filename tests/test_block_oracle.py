"""The oracle of the operators around the FFN, pinned on the CPU: published
generator outputs, closed forms, differences, a library's conversions."""

import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("counter,key,want", [
    # known answers that Random123, the generator's own distribution, is tested with
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert O.philox4x32(counter, key) == want


def test_keep_mask_bits_and_rate():
    m = O.keep_mask(3, 19, 0.5, 7, (5 << 32) + 6)
    w = O.philox4x32((1, 2, 6, 5), (7, 0))
    assert [bool(m[2, 8 + j]) for j in range(8)] == [
        ((w[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= 32768 for j in range(8)]
    assert O.keep_mask(2, 8, 0.0, 1, 1).all()
    big = O.keep_mask(64, 512, 0.1, 123, 0)
    n = big.size  # 5 standard deviations of the count of a fair draw
    assert abs((~big).sum() - 0.1 * n) < 5 * np.sqrt(n * 0.1 * 0.9)
    assert (O.keep_mask(8, 64, 0.3, 1, 0) != O.keep_mask(8, 64, 0.3, 1, 1)).any()
    assert (O.keep_mask(8, 64, 0.3, 1, 0) != O.keep_mask(8, 64, 0.3, 2, 0)).any()


def test_dropout_is_unbiased_and_zero_where_dropped():
    x = np.ones((64, 256))
    x[0, :] = np.inf
    y = O.dropout(x, 0.25, 3, 9)
    keep = O.keep_mask(64, 256, 0.25, 3, 9)
    assert (y[~keep] == 0).all() and np.allclose(y[1:][keep[1:]], 4 / 3)
    assert abs(y[1:].mean() - 1) < 5 * np.sqrt(1 / 3 / (63 * 256))


def test_rmsnorm_closed_forms():
    n, r = O.rmsnorm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([1.0, 2.0]), 0.0 + 1e-300)
    assert np.allclose(r[0], 1 / np.sqrt(12.5)) and np.allclose(n[0], [3 / np.sqrt(12.5), 8 / np.sqrt(12.5)])
    rng = np.random.default_rng(1)
    s = rng.standard_normal((4, 31))
    n, _ = O.rmsnorm(s, np.ones(31), 0.0)
    assert np.allclose((n * n).mean(axis=1), 1)
    assert np.allclose(O.rmsnorm(5 * s, np.ones(31), 0.0)[0], n)  # scale-free without eps


@pytest.mark.parametrize("d", [1, 5, 32])
def test_rmsnorm_gradient_against_differences(d):
    rng = np.random.default_rng(d)
    s, w, g = rng.standard_normal((3, d)), rng.standard_normal(d), rng.standard_normal((3, d))
    eps = 0.1
    ds, dw = O.rmsnorm_backward(g, s, w, O.rmsnorm(s, w, eps)[1])
    for v, grad, f in ((s, ds, lambda a: O.rmsnorm(a, w, eps)[0]), (w, dw, lambda a: O.rmsnorm(s, a, eps)[0])):
        u = rng.standard_normal(v.shape)
        t = 1e-6
        diff = ((f(v + t * u) - f(v - t * u)) * g).sum() / (2 * t)
        assert abs(diff - (grad * u).sum()) < 1e-7 * (1 + abs(diff))


def test_e4m3_values_against_torch():
    torch = pytest.importorskip("torch")
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_values(), want, equal_nan=True)
    # a byte of sign and a magnitude of 0..15 is an integer in units of 2^-9
    v = O.e4m3_values() * 512
    assert [v[m] for m in range(16)] == list(range(16)) and [v[128 + m] for m in range(16)] == [-m for m in range(16)]


def test_codes_and_dequantization():
    q = np.array([[1, 2, 3], [15, 0, 8]], dtype=np.uint8)
    assert O.pack_codes(q).tolist() == [[0x21, 0x03], [0x0F, 0x08]]
    s = np.array([[0.5, 2.0], [1.0, 1.0]])
    z = np.array([[1, 3], [0, 15]], dtype=np.uint8)
    assert O.q4_dequantize(q, s, None, 2).tolist() == [[-3.5, -3.0, -10.0], [7.0, -8.0, 0.0]]
    assert O.q4_dequantize(q, s, z, 2).tolist() == [[0.0, 0.5, 0.0], [15.0, 0.0, -7.0]]


def test_quantize_is_nearest():
    rng = np.random.default_rng(5)
    W = O.decode_bf16((rng.integers(0x3C00, 0x4000, (7, 100)) | (rng.integers(0, 2, (7, 100)) << 15)).astype(np.uint16))
    W[3, 64:] = 0
    codes, scales = O.q4_quantize(W, 32)
    back = O.q4_dequantize(codes, scales, None, 32)
    g = np.arange(100) // 32
    # half a step, and at the group's largest value what rounding the scale to bf16 moves 7 steps by
    assert (np.abs(back - W) <= scales[:, g] * (0.5 + 7 * 2.0**-8)).all()
    assert (codes[3, 64:] == 8).all() and (scales[3, 2:] == 0).all()


def test_gated_hidden():
    x = np.array([[1.0, -1.0]])
    h = O.gated_hidden(x, np.array([[2.0, 1.0], [1.0, 1.0], [0.0, 1.0]]), np.array([[3.0, 0.0]] * 3))
    assert h.tolist() == [[3.0, 0.0, 0.0]]
