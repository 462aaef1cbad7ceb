"""The oracle of layer norm, the adapters and the optimizer's step, pinned on the
CPU: closed forms, differences, a library's optimizer and conversions."""

import numpy as np
import pytest

import oracle as O


def test_layernorm_closed_forms():
    n, mean, rstd = O.layernorm(np.array([[1.0, 3.0], [5.0, 5.0]]), np.array([1.0, 2.0]), np.array([0.5, 0.0]), 1e-12)
    assert np.allclose(mean, [2, 5]) and np.allclose(rstd, [1, 1e6]) and np.allclose(n, [[-0.5, 2.0], [0.5, 0.0]])
    rng = np.random.default_rng(1)
    s = rng.standard_normal((4, 31))
    n, _, _ = O.layernorm(s, np.ones(31), None, 0.0)
    assert np.allclose(n.mean(axis=1), 0) and np.allclose((n * n).mean(axis=1), 1)
    assert np.allclose(O.layernorm(5 * s + 3, np.ones(31), None, 0.0)[0], n)  # free of scale and shift without eps


@pytest.mark.parametrize("d", [1, 5, 32])
def test_layernorm_gradient_against_differences(d):
    rng = np.random.default_rng(d)
    s, w, b, g = rng.standard_normal((3, d)), rng.standard_normal(d), rng.standard_normal(d), rng.standard_normal((3, d))
    eps = 0.1
    _, mean, rstd = O.layernorm(s, w, b, eps)
    ds, dw, db = O.layernorm_backward(g, s, w, mean, rstd)
    for v, grad, f in ((s, ds, lambda a: O.layernorm(a, w, b, eps)[0]), (w, dw, lambda a: O.layernorm(s, a, b, eps)[0]),
                       (b, db, lambda a: O.layernorm(s, w, a, eps)[0])):
        u = rng.standard_normal(v.shape)
        t = 1e-6
        diff = ((f(v + t * u) - f(v - t * u)) * g).sum() / (2 * t)
        assert abs(diff - (grad * u).sum()) < 1e-7 * (1 + abs(diff))


def test_lora_is_a_sum_of_products():
    rng = np.random.default_rng(2)
    x, A, B = rng.standard_normal((5, 7)), rng.standard_normal((3, 2, 7)), rng.standard_normal((3, 4, 2))
    base, scaling = rng.standard_normal((5, 4)), np.array([1.0, 0.5, 2.0])
    y = O.lora(x, np.array([2, -1, 0, 3, 2]), A, B, scaling, base)
    assert np.array_equal(y[[1, 3]], base[[1, 3]])
    for m, a in ((0, 2), (2, 0), (4, 2)):
        want = base[m] + scaling[a] * sum(B[a][:, r] * (A[a][r] * x[m]).sum() for r in range(2))
        assert np.allclose(y[m], want)


def test_adamw_against_a_library():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    p0 = rng.standard_normal(50)
    q = torch.from_numpy(p0.copy()).requires_grad_()
    opt = torch.optim.AdamW([q], lr=3e-2, betas=(0.8, 0.95), eps=1e-3, weight_decay=0.2)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        q.grad = torch.from_numpy(g.copy()) * 0.5
        opt.step()
        p, m, v = O.adamw(p, g, m, v, step, 3e-2, 0.8, 0.95, 1e-3, 0.2, 0.5)
        assert np.allclose(p, q.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_to_neighbour():
    rng = np.random.default_rng(4)
    grid = O.e4m3_values()[:127]
    bits = np.arange(256)
    for v in grid:  # what e4m3 holds stays as it is, with either sign
        assert (O.to_neighbour(np.full(256, v), bits) == v).all() and (O.to_neighbour(np.full(256, -v), bits) == -v).all()
    for lo, hi in zip(grid[:-1], grid[1:]):  # a quarter of the way up: a quarter of the draws
        q = O.to_neighbour(np.full(256, lo + (hi - lo) / 4), bits)
        assert set(np.unique(q)) == {lo, hi} and (q == hi).sum() == 64
    x = rng.uniform(-448, 448, 1000)
    q = O.to_neighbour(x, rng.integers(0, 256, 1000))
    assert (np.abs(q - x) <= np.maximum(np.abs(x) / 8, 2.0**-9)).all() and (np.sign(q) * np.sign(x) >= 0).all()
    assert (O.to_neighbour(np.array([1e-30, 0.0]), np.zeros(2), 2.0**-9) == [2.0**-9, 0.0]).all()


def test_state_bits_and_scales():
    bits = O.state_bits(19, 5, 7, (3 << 32) + 9)
    w = O.philox4x32((2, 5, 9, 3), (7, 0))
    assert bits[16] == w[0] & 0xFFFF and bits[17] == w[0] >> 16 and bits[18] == w[1] & 0xFFFF and len(bits) == 19
    v = np.arange(600.0) - 300
    assert np.allclose(O.block_scales(v) * 448, [300, 211, 299]) and (O.block_scales(np.zeros(3)) * 448 == 2.0**-100).all()
