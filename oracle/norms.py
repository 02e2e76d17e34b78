"""CPU oracle of the layer norms with one scale and shift per group of a packed
batch, with their backward pass, and of the norms and clipping of gradients
over many tensors (binary64 numpy).

TEST INFRASTRUCTURE ONLY: the plain, slow definitions the GPU kernels are
checked against; it imports nothing from the GPU package.

Layer norm: with m, v the mean and variance of a row's C values, s = (v +
eps)^-1/2 and h = s (x - m), for the rows r of group n
    y_r = gamma_n h_r + beta_n;  q = gamma_n g_r,
    grad_x_r = s (q - mean q - h_r mean(q h_r)),
    grad_gamma_n = sum_r g_r h_r,  grad_beta_n = sum_r g_r.

Clipping: n_g = sqrt(sum v^2) over group g's slices of all tensors, out = v
min(1, max_norm / (n_g + eps)).
"""

from __future__ import annotations

import numpy as np

from .grouped_linear import TINY, UNIT, sum_error_bound

# of a binary32 operation, with one more bit than a correct rounding needs
ROUND = 2.0 ** -23


def _group_of(row_offsets, rows):
    return np.searchsorted(np.asarray(row_offsets, np.int64)[1:], np.arange(rows), side="right")


def _normalised(x, eps):
    x = np.asarray(x, np.float64)
    centred = x - x.mean(axis=1, keepdims=True)
    s = 1.0 / np.sqrt((centred * centred).mean(axis=1, keepdims=True) + eps)
    return centred * s, s


def _rows_of(values, row_offsets, shape, fill):
    if values is None:
        return np.full(shape, fill)
    return np.asarray(values, np.float64)[_group_of(row_offsets, shape[0])]


def layer_norm_forward(x, row_offsets, weight=None, bias=None, eps=1e-5):
    """x [R, C], weight and bias [N, C] -> y [R, C]."""
    h, _ = _normalised(x, eps)
    return h * _rows_of(weight, row_offsets, h.shape, 1.0) + _rows_of(bias, row_offsets, h.shape, 0.0)


def layer_norm_backward(x, row_offsets, weight, grad_y, eps=1e-5):
    """(grad_x, grad_weight, grad_bias) from grad_y [R, C]."""
    h, s = _normalised(x, eps)
    g = np.asarray(grad_y, np.float64)
    q = g * _rows_of(weight, row_offsets, h.shape, 1.0)
    gx = s * (q - q.mean(axis=1, keepdims=True) - h * (q * h).mean(axis=1, keepdims=True))
    off = np.asarray(row_offsets, np.int64)
    gw = np.stack([(g * h)[a:b].sum(axis=0) for a, b in zip(off, off[1:])]) if len(off) > 1 else np.zeros((0, h.shape[1]))
    gb = np.stack([g[a:b].sum(axis=0) for a, b in zip(off, off[1:])]) if len(off) > 1 else np.zeros((0, h.shape[1]))
    return gx, gw, gb


def _h_error(x, eps):
    """Bounds on the error of h and the relative error of s, with every
    operation off by at most u = ROUND of its result.

    The mean m' is off by at most e = (C + 1) u mean|x|. The deviations d' from
    it are rounded once (u |d'|); their mean, which is m - m' but for rounding,
    is off by (C + 2) u mean|d'|, and mean|d'| is at most D = sqrt(v) + e; so
    the numerator d' - mean d' is off by u (2 |d| + (C + 4) D). The variance
    mean d'^2 - (mean d')^2 is off by (C + 6) u D^2, which moves s by half of
    that over v + eps, relatively; sum, root and reciprocal round it 4 times."""
    x = np.asarray(x, np.float64)
    C = x.shape[1]
    h, s = _normalised(x, eps)
    centred = h / s
    v = (centred * centred).mean(axis=1, keepdims=True)
    D = np.sqrt(v) + (C + 1) * ROUND * np.abs(x).mean(axis=1, keepdims=True)
    rel = 0.5 * (C + 6) * ROUND * D * D * s * s + 4 * ROUND
    return s * ROUND * (2 * np.abs(centred) + (C + 4) * D) + np.abs(h) * rel, rel


def _stored(error, value, dtype):
    return error + UNIT[dtype] * (np.abs(value) + error) + TINY[dtype]


def layer_norm_forward_bound(x, row_offsets, weight, bias, dtype, eps=1e-5):
    y = layer_norm_forward(x, row_offsets, weight, bias, eps)
    gamma = np.abs(_rows_of(weight, row_offsets, y.shape, 1.0))
    e, _ = _h_error(x, eps)
    h, _ = _normalised(x, eps)
    return _stored(gamma * e + ROUND * (gamma * np.abs(h) + np.abs(y)), y, dtype)


def layer_norm_backward_bound(x, row_offsets, weight, grad_y, dtype, eps=1e-5):
    """As for the sums of grouped_linear.sum_error_bound, with h's error beside them."""
    x, g = np.asarray(x, np.float64), np.asarray(grad_y, np.float64)
    C = x.shape[1]
    (h, s), (e, rel) = _normalised(x, eps), _h_error(x, eps)
    q = np.abs(g * _rows_of(weight, row_offsets, h.shape, 1.0))
    value = layer_norm_backward(x, row_offsets, weight, grad_y, eps)
    mean = lambda t: t.mean(axis=1, keepdims=True)  # noqa: E731
    mq, mh = mean(q), mean(q * np.abs(h))
    mh_error = (C + 3) * ROUND * mh + mean(q * e)
    t_error = (C + 2) * ROUND * mq + np.abs(h) * mh_error + (mh + mh_error) * e + 4 * ROUND * (q + mq + np.abs(h) * mh)
    gx = s * (1 + rel) * t_error + np.abs(value[0]) * rel
    off = np.asarray(row_offsets, np.int64)
    rows = np.diff(off).astype(np.float64)[:, None]
    sums = lambda t: np.stack([t[a:b].sum(axis=0) for a, b in zip(off, off[1:])])  # noqa: E731
    gw = sum_error_bound(sums(np.abs(g * h)), rows, value[1], dtype) + (1 + UNIT[dtype]) * sums(np.abs(g) * e)
    return _stored(gx, value[0], dtype), gw, sum_error_bound(sums(np.abs(g)), rows, value[2], dtype)


def clip_grad_norm(tensors, max_norm, groups=1, eps=1e-6):
    """([clipped tensors], norms [groups]); each tensor has groups equal slices."""
    flat = [np.asarray(t, np.float64).reshape(groups, -1) for t in tensors]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        norms = np.sqrt(sum((f * f).sum(axis=1) for f in flat))
        factor = np.minimum(1.0, max_norm / (norms + eps))
        factor = np.where(norms + eps == 0.0, 1.0, factor)
        return [(f * factor[:, None]).reshape(np.shape(t)) for f, t in zip(flat, tensors)], norms


def clip_bound(value, dtype):
    """Factor and product are rounded to binary32, then to the type (the same rounding for float32)."""
    value = np.abs(value)
    return value * (2.0 ** -24 + UNIT["float32"] + (0.0 if dtype == "float32" else UNIT[dtype])) * (1 + 2.0 ** -8) + TINY[dtype]
