"""CPU oracle of the gated layers with one pair of weights per group of a
packed batch, and their backward pass (binary64 numpy).

TEST INFRASTRUCTURE ONLY: the plain, slow definition the GPU layer is checked
against; it imports nothing from the GPU package.

For the rows r of group n, weight [N, 2, F, C] = (A, U) and bias [N, 2, F]:
    a = A_n x_r + a_n,  u = U_n x_r + u_n,  y_r = act(a) u;
    da = g_r u act'(a),  du = g_r act(a),
    grad_x_r = A_n^T da + U_n^T du,  grad_weight_n = sum_r (da x_r^T, du x_r^T),
    grad_bias_n = sum_r (da, du).
"""

from __future__ import annotations

import math

import numpy as np

from .grouped_linear import TINY, UNIT, _groups, sum_error_bound

ROUND = 2.0 ** -23
K = math.sqrt(2.0 / math.pi)
ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "sigmoid")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _logistic(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def activate(a, kind):
    """(act(a), act'(a), the derivative's part that does not vanish with a)"""
    a = np.asarray(a, np.float64)
    if kind == "sigmoid":
        s = _logistic(a)
        return s, s * _logistic(-a), s * _logistic(-a)
    if kind == "gelu":
        below = 0.5 * (_erfc(-a / math.sqrt(2.0)) if a.size else a)
        return a * below, below + a * np.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi), below
    if kind == "silu":
        z, dz = a, 1.0
    elif kind == "gelu_tanh":
        z, dz = 2 * K * (a + 0.044715 * a ** 3), 2 * K * (1 + 3 * 0.044715 * a * a)
    else:
        raise ValueError(kind)
    s = _logistic(z)
    return a * s, s + a * s * _logistic(-z) * dz, s


def curvature(a, kind):
    """act''(a)"""
    a = np.asarray(a, np.float64)
    if kind == "gelu":
        return (2 - a * a) * np.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    z, dz, ddz = (2 * K * (a + 0.044715 * a ** 3), 2 * K * (1 + 3 * 0.044715 * a * a), 2 * K * 6 * 0.044715 * a) \
        if kind == "gelu_tanh" else (a, 1.0, 0.0)
    s, p = _logistic(z), _logistic(z) * _logistic(-z)
    if kind == "sigmoid":
        return p * (1 - 2 * s)
    return 2 * p * dz + a * p * ((1 - 2 * s) * dz * dz + ddz)


def _projections(x, row_offsets, weight, bias):
    N, _, F, C = weight.shape
    both = np.zeros((x.shape[0], 2, F))
    for n, rows in _groups(row_offsets):
        both[rows] = (x[rows] @ weight[n].reshape(2 * F, C).T).reshape(rows.stop - rows.start, 2, F)
        if bias is not None:
            both[rows] += bias[n]
    return both[:, 0], both[:, 1]


def _doubles(*arrays):
    return tuple(None if v is None else np.asarray(v, np.float64) for v in arrays)


def gated_forward(x, row_offsets, weight, bias=None, activation="silu"):
    x, weight, bias = _doubles(x, weight, bias)
    a, u = _projections(x, row_offsets, weight, bias)
    return activate(a, activation)[0] * u


def gated_backward(x, row_offsets, weight, bias, grad_y, activation="silu"):
    """(grad_x, grad_weight, grad_bias) from grad_y [R, F]."""
    x, weight, bias, g = _doubles(x, weight, bias, grad_y)
    a, u = _projections(x, row_offsets, weight, bias)
    act, slope, _ = activate(a, activation)
    return _products(x, row_offsets, weight, np.stack([g * u * slope, g * act], axis=1))


def _products(x, row_offsets, weight, back):
    gx, gw, gb = np.zeros_like(x), np.zeros_like(weight), np.zeros(weight.shape[:3])
    for n, rows in _groups(row_offsets):
        flat = back[rows].reshape(rows.stop - rows.start, 2 * weight.shape[2])
        gx[rows] = flat @ weight[n].reshape(flat.shape[1], x.shape[1])
        gw[n] = (flat.T @ x[rows]).reshape(gw[n].shape)
        gb[n] = back[rows].sum(axis=0)
    return gx, gw, gb


def activation_error(a, kind, known=None):
    """Bounds on the errors of act(a) and act'(a) as they are evaluated in binary32 from a itself.

    u = ROUND is the error of a hardware exponential or reciprocal, and of two
    correct roundings. An exponential e^-z, z formed with r roundings, is off by
    2 u and r u / 2 times z, relatively: E. The logistic function s = 1 / (1 +
    e^-z) by (1 - s) E + 3 u, and nothing where e^-z vanishes beside 1.
    silu, gelu_tanh (v = a s, v' = s + v (1 - s) z'): r is 2 and 5; 1 - s is off
    by what s is, and a rounding. sigmoid (s and e s^2 of the magnitude; below
    zero e s): r is 2. gelu: the tail t Q(t) e^(-a^2 / 2) beyond |a|, with t and
    Q off by 8 u together and the exponential's argument by 3 roundings; the
    derivative is a e^(-a^2 / 2) / sqrt(2 pi) + its normal distribution.
    Exponentials below 2^-126 may vanish."""
    a = np.asarray(a, np.float64)
    value, slope, first = known or activate(a, kind)
    m, gone = np.abs(a), 2.0 ** -125 * (1 + np.abs(a))
    if kind == "sigmoid":
        e, s = (2 + m) * ROUND, _logistic(m)
        es = (1 - s) * e + 3 * ROUND
        return np.abs(value) * (np.where(a < 0, e, 0.0) + es + ROUND) + gone, slope * (e + 2 * es + 2 * ROUND) + gone
    if kind == "gelu":
        e = (2 + 0.75 * a * a) * ROUND
        tail = np.minimum(first, 0.5 * np.exp(-0.5 * a * a)) * (e + 10 * ROUND)   # of the distribution below -|a|, or a bound
        below = tail + ROUND * first
        return m * below + ROUND * np.abs(value) + gone, below + np.abs(slope - first) * (e + 2 * ROUND) + ROUND * np.abs(slope) + gone
    r, z, dz = (2, a, 1.0) if kind == "silu" else (5, 2 * K * (a + 0.044715 * a ** 3), 2 * K * (1 + 3 * 0.044715 * a * a))
    s, rest = _logistic(z), _logistic(-z)
    es = np.where(rest < 2.0 ** -25, rest, rest * (2 + 0.5 * r * np.abs(z)) * ROUND + 3 * ROUND)    # relative
    eslope = s * es + np.abs(value) * dz * (s * es + ROUND * rest + rest * (es + 6 * ROUND)) + ROUND * np.abs(slope)
    return np.abs(value) * (es + ROUND) + gone, eslope + gone * (1 + dz)    # a vanished s in a s z'


def _parts(x, row_offsets, weight, bias, activation):
    """a, u, act(a), act'(a), and bounds on the error of each.

    a and u are sums of C + 1 products in binary32: (C + 3) u of the sum of
    absolute values, u = ROUND: e. act moves with a by its derivative there, and
    1/2 e^2 times the second, which is at most 1 in magnitude; act' by the second,
    and the third is at most 2. Their own evaluation
    (activation_error) is at a value of a that is e off: a hundredth more."""
    a, u = _projections(x, row_offsets, weight, bias)
    mag = _projections(np.abs(x), row_offsets, np.abs(weight), None if bias is None else np.abs(bias))
    ea, eu = ((x.shape[1] + 3) * ROUND * m for m in mag)
    act, slope, _ = known = activate(a, activation)
    own_act, own_slope = activation_error(a, activation, known)
    eact = 1.01 * (own_act + np.abs(slope) * ea + 0.5 * ea * ea)
    eslope = 1.01 * (own_slope + np.abs(curvature(a, activation)) * ea + ea * ea)
    return a, u, act, slope, eu, eact, eslope


def gated_forward_bound(x, row_offsets, weight, bias, dtype, activation="silu"):
    x, weight, bias = _doubles(x, weight, bias)
    _, u, act, _, eu, eact, _ = _parts(x, row_offsets, weight, bias, activation)
    y = act * u
    e = np.abs(u) * eact + np.abs(act) * eu + eact * eu + ROUND * np.abs(y)
    return e + UNIT[dtype] * (np.abs(y) + e) + TINY[dtype]


# what [da du] is off by as it enters its products, relatively: a rounding to
# float32; the rest of a pair of bfloat16 (each part off by half a step, 2^-8 of
# it, at most); with float16 operands as much again for low times low, which is left out
HELD = {"float32": UNIT["float32"], "float16": 2.0 ** -15, "bfloat16": 2.0 ** -16}
PRODUCTS = {"float32": 1, "float16": 3, "bfloat16": 2}     # of a term, each added


def gated_backward_bound(x, row_offsets, weight, bias, grad_y, dtype, activation="silu"):
    """[da du] with the errors of its factors and as it is held, then sums as for linear layers."""
    x, weight, bias, g = _doubles(x, weight, bias, grad_y)
    _, u, act, slope, eu, eact, eslope = _parts(x, row_offsets, weight, bias, activation)
    da, du = g * u * slope, g * act
    ea = np.abs(g) * (np.abs(u) * eslope + np.abs(slope) * eu + eslope * eu) + 2 * ROUND * np.abs(da)
    ed = np.abs(g) * eact + ROUND * np.abs(du)
    back, eback = np.stack([da, du], axis=1), np.stack([ea, ed], axis=1)
    eback = eback + HELD[dtype] * (np.abs(back) + eback) + 2.0 ** -126   # no type's range but float32's
    value = _products(x, row_offsets, weight, back)
    mag = _products(np.abs(x), row_offsets, np.abs(weight), np.abs(back) + eback)
    extra = _products(np.abs(x), row_offsets, np.abs(weight), eback)
    rows = np.diff(np.asarray(row_offsets, np.int64)).astype(np.float64)
    terms = tuple(PRODUCTS[dtype] * t for t in (2 * weight.shape[2], rows[:, None, None, None], rows[:, None, None]))
    return tuple(sum_error_bound(m, t, v, dtype) + (1 + UNIT[dtype]) * e for m, t, v, e in zip(mag, terms, value, extra))
