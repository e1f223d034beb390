"""Pins of oracle.block that use none of its own formulas: hand-worked values, gradients against
differences of the forward pass, rotations as complex products, torch's stable sort."""

import numpy as np
import pytest
import torch

from oracle import block as ob
from oracle import e4m3


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).double().numpy()


def test_norm_of_a_worked_row():
    # h = (3, 4, 0, ...): mean square 25 / 128, y = h / (5 / sqrt(128)) with eps -> 0
    x = np.zeros((1, 128))
    x[0, :2] = 3.0, 4.0
    h, y = ob.add_rmsnorm(x, None, np.ones(128), 1e-30)
    assert np.allclose(y[0, :2], np.array([0.6, 0.8]) * np.sqrt(128), rtol=1e-14)
    codes, S = ob.quant_rows(h, np.ones(128), y)
    # 4 is the group's largest: code of 448; 3 becomes 336 = 1.3125 * 2^8, a tie between 320 and
    # 352 that goes to the even mantissa 320 (1.25 * 2^8, mantissa 2)
    assert list(e4m3.decode(codes[0, :3])) == [320.0, 448.0, 0.0]
    assert np.allclose(S, 0.8 * np.sqrt(128) / 448)


def test_stream_rounding_is_one_rounding_of_the_exact_sum():
    rng = np.random.default_rng(3)
    x = bf16(rng, 400, 128) * 2.0 ** rng.integers(-40, 40, (400, 128))
    r = bf16(rng, 400, 128) * 2.0 ** rng.integers(-40, 40, (400, 128))
    h, _ = ob.add_rmsnorm(x, r, np.ones(128), 1e-6)
    two = (x.astype(np.float32) + r.astype(np.float32))
    want = torch.from_numpy(two).to(torch.bfloat16).double().numpy()
    assert np.array_equal(h, want)


def test_norm_gradients_match_differences():
    rng = np.random.default_rng(4)
    M, K, eps = 3, 128, 1e-3
    h, w, dy, dh = bf16(rng, M, K), bf16(rng, K), bf16(rng, M, K), bf16(rng, M, K)

    def loss(h, w):
        y = h * w / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
        return float((y * dy).sum() + (h * dh).sum())

    dx, dw, _, _ = ob.add_rmsnorm_bwd(dy, h, w, dh, eps)
    s = 1e-6
    for m, k in ((0, 0), (1, 17), (2, 127)):
        e = np.zeros_like(h)
        e[m, k] = s
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * s) - dx[m, k]) < 1e-6
    for k in (0, 5, 127):
        e = np.zeros_like(w)
        e[k] = s
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * s) - dw[k]) < 1e-6


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (7, 3, 5), (50, 8, 16)])
def test_sort_agrees_with_a_stable_sort(T, k, E):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E + 1, (T, k))
    off, rows, pos = ob.moe_sort(ids, E)
    flat = torch.from_numpy(ids.reshape(-1))
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices.numpy()
    n = int((key < E).sum())
    assert off[E] == n and list(rows[:n]) == list(order[:n] // k) and np.all(rows[n:] == -1)
    assert list(pos.reshape(-1)[order[:n]]) == list(range(n))
    assert int((pos >= 0).sum()) == n
    assert list(np.diff(off)) == [int((key == e).sum()) for e in range(E)]


def test_combine_and_its_gradient_by_differences():
    rng = np.random.default_rng(6)
    y, w, dout = bf16(rng, 6, 8), rng.standard_normal((3, 2)), bf16(rng, 3, 8)
    pos = np.array([[0, 3], [5, -1], [2, 1]])
    out, _ = ob.moe_combine(y, pos, w)
    assert np.allclose(out[1], w[1, 0] * y[5])
    d, _ = ob.moe_dweights(dout, y, pos)
    for t, j in ((0, 0), (0, 1), (1, 0), (1, 1), (2, 1)):
        e = np.zeros_like(w)
        e[t, j] = 1.0
        diff = (ob.moe_combine(y, pos, w + e)[0] - out) * dout  # the sum is linear in w
        assert abs(diff.sum() - d[t, j]) < 1e-12


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(7)
    x, ang = rng.standard_normal((5, 48)), rng.standard_normal((5, 16))
    out, _ = ob.rope(x, None, 0.0, np.cos(ang), np.sin(ang), 32, interleaved)
    a = slice(0, 32, 2) if interleaved else slice(0, 16)
    b = slice(1, 32, 2) if interleaved else slice(16, 32)
    z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * ang)
    assert np.allclose(out[:, a], z.real) and np.allclose(out[:, b], z.imag)
    assert np.array_equal(out[:, 32:], x[:, 32:])
