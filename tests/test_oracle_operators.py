"""Pins of the oracles of the per-group linear layers (oracle/grouped_linear.py)
and the orthogonalised updates (oracle/orthogonalize.py): hand-worked cases,
finite differences, invariants, and planted mistakes that the pins must see."""

import numpy as np
import pytest

from oracle.grouped_linear import (backward_error_bound, forward_error_bound, grouped_linear_backward,
                                   grouped_linear_forward)
from oracle.orthogonalize import amplification, expected_error, orthogonalize, polynomial


def test_layer_hand_case():
    # two groups of 2 and 1 rows with an empty one between
    x = np.array([[1.0, 2.0], [0.0, -1.0], [3.0, 0.5]])
    w = np.array([[[1.0, 0.0], [2.0, 1.0], [0.0, -1.0]], np.full((3, 2), 9.0), [[0.0, 2.0], [1.0, 1.0], [4.0, 0.0]]])
    b = np.array([[0.0, 1.0, 0.5], [7.0, 7.0, 7.0], [0.0, 0.0, -1.0]])
    y = grouped_linear_forward(x, [0, 2, 2, 3], w, b)
    np.testing.assert_array_equal(y, [[1.0, 5.0, -1.5], [0.0, 0.0, 1.5], [1.0, 3.5, 11.0]])
    g = np.array([[1.0, 0.0, 2.0], [0.0, 1.0, 0.0], [1.0, 1.0, 0.0]])
    gx, gw, gb = grouped_linear_backward(x, [0, 2, 2, 3], w, g)
    np.testing.assert_array_equal(gx, [[1.0, -2.0], [2.0, 1.0], [1.0, 3.0]])
    np.testing.assert_array_equal(gw[0], [[1.0, 2.0], [0.0, -1.0], [2.0, 4.0]])
    np.testing.assert_array_equal(gw[1], np.zeros((3, 2)))
    np.testing.assert_array_equal(gw[2], [[3.0, 0.5], [3.0, 0.5], [0.0, 0.0]])
    np.testing.assert_array_equal(gb, [[1.0, 1.0, 2.0], [0.0, 0.0, 0.0], [1.0, 1.0, 0.0]])


def test_layer_gradient_is_the_finite_difference():
    rng = np.random.default_rng(1)
    off = [0, 3, 3, 4, 9]
    x, w, b = rng.normal(size=(9, 5)), rng.normal(size=(4, 3, 5)), rng.normal(size=(4, 3))
    g = rng.normal(size=(9, 3))
    grads = grouped_linear_backward(x, off, w, g)
    h = 1e-6
    for k, arr in enumerate((x, w, b)):
        for i in np.ndindex(arr.shape):
            up, down = arr.copy(), arr.copy()
            up[i] += h
            down[i] -= h
            args = [x, w, b]
            args[k] = up
            hi = np.sum(g * grouped_linear_forward(args[0], off, args[1], args[2]))
            args[k] = down
            lo = np.sum(g * grouped_linear_forward(args[0], off, args[1], args[2]))
            # the layer is linear in each argument: only rounding is left
            assert abs((hi - lo) / (2 * h) - grads[k][i]) < 1e-7


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_layer_error_bound_sees_a_missing_term(dtype):
    # a product left out of a short sum is far outside the bound
    rng = np.random.default_rng(2)
    off = [0, 5, 12]
    x, w, b = rng.normal(size=(12, 8)) + 3.0, rng.normal(size=(2, 4, 8)) + 3.0, rng.normal(size=(2, 4))
    y = grouped_linear_forward(x, off, w, b)
    bound = forward_error_bound(x, off, w, b, dtype)
    less = grouped_linear_forward(x[:, :7], off, w[:, :, :7], b)
    assert (np.abs(less - y) > bound).mean() > 0.9
    g = rng.normal(size=(12, 4)) + 3.0
    bounds = backward_error_bound(x, off, w, g, dtype)
    right = grouped_linear_backward(x, off, w, g)
    wrong = grouped_linear_backward(x[1:], [0, 4, 11], w, g[1:])     # the first row left out
    assert (np.abs(wrong[1][0] - right[1][0]) > bounds[1][0]).mean() > 0.9
    assert (np.abs(wrong[2][0] - right[2][0]) > bounds[2][0]).mean() > 0.9


def test_orthogonalize_hand_case():
    # one entry: X_0 = 1 (eps aside), p(1) = 0.701, and so on; both signs
    p = 3.4445 - 4.7750 + 2.0315
    np.testing.assert_allclose(orthogonalize([[2.0]], 1, 1e-30), [[p]], rtol=1e-14)
    np.testing.assert_allclose(orthogonalize([[-2.0]], 2, 1e-30), [[-(3.4445 * p - 4.775 * p ** 3 + 2.0315 * p ** 5)]],
                               rtol=1e-14)
    np.testing.assert_array_equal(orthogonalize(np.zeros((2, 3))), np.zeros((2, 3)))


@pytest.mark.parametrize("m,n", [(4, 4), (3, 9), (9, 3)])
def test_orthogonalize_keeps_the_singular_vectors(m, n):
    rng = np.random.default_rng(m * 10 + n)
    u = rng.normal(size=(m, n))
    left, s, right = np.linalg.svd(u, full_matrices=False)
    s0 = s / (np.linalg.norm(u) + 1e-7)
    want = (left * polynomial(s0, 5)[0]) @ right
    np.testing.assert_allclose(orthogonalize(u), want, atol=1e-12)
    # the same matrix transposed: X X^T and X^T X lead to the same iteration
    np.testing.assert_allclose(orthogonalize(u.T), want.T, atol=1e-12)
    x = orthogonalize(u)
    assert np.abs(np.linalg.svd(x, compute_uv=False) - 1.0).max() < 0.5


@pytest.mark.parametrize("m,n", [(5, 7), (6, 6), (1, 4)])
def test_amplification_is_the_finite_difference(m, n):
    rng = np.random.default_rng(7)
    u = rng.normal(size=(m, n))
    x = u / np.linalg.norm(u)

    def run(v):
        for _ in range(3):
            g = v @ v.T
            v = 3.4445 * v + (-4.7750 * g + 2.0315 * g @ g) @ v
        return v

    # mean over a basis of perturbations: exact up to the difference quotient
    total = 0.0
    for i in np.ndindex(m, n):
        e = np.zeros((m, n))
        e[i] = 1e-6
        total += np.sum(((run(x + e) - run(x - e)) / 2e-6) ** 2)
    amp = amplification(np.linalg.svd(x, compute_uv=False), n, 3)
    np.testing.assert_allclose(amp, np.sqrt(total / (m * n)), rtol=1e-6)


def _rounded(update, bits, steps=5):
    """The iteration with every factor of a product rounded to `bits` bits."""
    def cut(v):
        mant, ex = np.frexp(v)
        return np.ldexp(np.round(np.ldexp(mant, bits)), ex - bits)

    x = update / np.linalg.norm(update)
    for _ in range(steps):
        g = cut(x) @ cut(x).T
        x = 3.4445 * x + cut(-4.7750 * g + 2.0315 * cut(g) @ cut(g)) @ cut(x)
    return x


@pytest.mark.parametrize("m,n", [(3, 64), (24, 40), (64, 64)])
def test_expected_error_is_that_of_rounded_factors(m, n):
    u = np.random.default_rng(m).normal(size=(m, n))
    x = orthogonalize(u, 5, 1e-30)
    for bits in (11, 16, 20):
        got = np.linalg.norm(_rounded(u, bits) - x)
        want = expected_error(u, 5, 1e-30, 2.0 ** -(bits + 1), 0.0)
        assert want / 12 < got < 2 * want


@pytest.mark.parametrize("unit,out", [(2.0 ** -23, 2.0 ** -24), (2.0 ** -12, 2.0 ** -8)])
def test_expected_error_sees_a_missing_step_and_a_wrong_coefficient(unit, out):
    u = np.random.default_rng(8).normal(size=(24, 40))
    x = orthogonalize(u)
    expect = expected_error(u, 5, 1e-7, unit, out)
    assert np.linalg.norm(orthogonalize(u, 4) - x) > 8 * expect
    v = u / np.linalg.norm(u)
    for _ in range(5):
        g = v @ v.T
        v = 3.4445 * v + (-4.7750 * g + 2.4 * g @ g) @ v
    assert np.linalg.norm(v - x) > 8 * expect
