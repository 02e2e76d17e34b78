"""CPU oracle of the linear layers with one weight per group of a packed
batch, and their backward pass (binary64 numpy).

TEST INFRASTRUCTURE ONLY: the plain, slow definition the GPU layer is checked
against; it imports nothing from the GPU package.

Group n owns rows [row_offsets[n], row_offsets[n+1]) and for its rows
    y_r = W_n x_r + b_n,
    grad_x_r = W_n^T g_r,  grad_W_n = sum_r g_r x_r^T,  grad_b_n = sum_r g_r.
"""

from __future__ import annotations

import numpy as np

# unit roundoff and smallest positive value of the storage types
UNIT = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -24, "bfloat16": 2.0 ** -133}


def _groups(row_offsets):
    off = np.asarray(row_offsets, np.int64)
    return [(n, slice(int(a), int(b))) for n, (a, b) in enumerate(zip(off, off[1:]))]


def grouped_linear_forward(x, row_offsets, weight, bias=None):
    """x [R, in], weight [N, out, in], bias [N, out] -> y [R, out]."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    y = np.zeros((x.shape[0], weight.shape[1]))
    for n, rows in _groups(row_offsets):
        y[rows] = x[rows] @ weight[n].T
        if bias is not None:
            y[rows] += np.asarray(bias, np.float64)[n]
    return y


def grouped_linear_backward(x, row_offsets, weight, grad_y):
    """(grad_x, grad_weight, grad_bias) from grad_y [R, out]."""
    x, weight, g = (np.asarray(v, np.float64) for v in (x, weight, grad_y))
    gx, gw = np.zeros_like(x), np.zeros_like(weight)
    gb = np.zeros(weight.shape[:2])
    for n, rows in _groups(row_offsets):
        gx[rows] = g[rows] @ weight[n]
        gw[n] = g[rows].T @ x[rows]
        gb[n] = g[rows].sum(axis=0)
    return gx, gw, gb


def sum_error_bound(magnitude, terms, value, dtype):
    """Bound on the error of a sum of `terms` products added in binary32 in any
    order (each product and each addition rounded by at most 2^-23 of the
    running magnitude, the sum of absolute values), stored in `dtype`."""
    add = (np.asarray(terms) + 2) * 2.0 ** -23 * magnitude
    return add + UNIT[dtype] * (np.abs(value) + add) + TINY[dtype]


def forward_error_bound(x, row_offsets, weight, bias, dtype):
    mag = grouped_linear_forward(np.abs(x), row_offsets, np.abs(weight), None if bias is None else np.abs(bias))
    return sum_error_bound(mag, weight.shape[2] + 1, grouped_linear_forward(x, row_offsets, weight, bias), dtype)


def backward_error_bound(x, row_offsets, weight, grad_y, dtype):
    mag = grouped_linear_backward(np.abs(x), row_offsets, np.abs(weight), np.abs(grad_y))
    val = grouped_linear_backward(x, row_offsets, weight, grad_y)
    rows = np.diff(np.asarray(row_offsets, np.int64)).astype(np.float64)
    terms = (weight.shape[1], rows[:, None, None], rows[:, None])
    return tuple(sum_error_bound(m, t, v, dtype) for m, t, v in zip(mag, terms, val))
