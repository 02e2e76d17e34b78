"""CPU oracle of the orthogonalised updates (binary64 numpy) and the
error to expect of computing them with rounded factors.

TEST INFRASTRUCTURE ONLY; it imports nothing from the GPU package.

    X_0 = U / (|U|_F + eps),  X <- a X + (b A + c A A) X,  A = X X^T,
so a singular value s of X_0 becomes p(p(...p(s))), p(s) = a s + b s^3 + c s^5,
and the singular vectors stay.
"""

from __future__ import annotations

import numpy as np

A, B, C = 3.4445, -4.7750, 2.0315


def orthogonalize(update, steps=5, eps=1e-7):
    """update [m, n] or [B, m, n] -> the same shape."""
    u = np.asarray(update, np.float64)
    if u.ndim == 3:
        return np.stack([orthogonalize(v, steps, eps) for v in u]) if len(u) else u
    x = u / (np.sqrt(np.sum(u * u)) + eps)
    for _ in range(steps):
        gram = x @ x.T
        x = A * x + (B * gram + C * gram @ gram) @ x
    return x


def polynomial(s, steps):
    """(value, derivative) of `steps` applications of p."""
    v, d = np.asarray(s, np.float64), np.ones_like(s, dtype=np.float64)
    for _ in range(steps):
        d = d * (A + 3 * B * v ** 2 + 5 * C * v ** 4)
        v = A * v + B * v ** 3 + C * v ** 5
    return v, d


def amplification(s, long_, steps):
    """Root mean square of the factors by which `steps` further steps stretch
    a small random perturbation (Frobenius norm) of a matrix [len(s), long_]
    of singular values s. X -> V f(S) W^T stretches the part of it between two
    singular directions by the divided differences (f(s) - f(t)) / (s - t)
    (symmetric) and (f(s) + f(t)) / (s + t) (antisymmetric), and the part
    outside the row space by f(s) / s."""
    s = np.maximum(np.asarray(s, np.float64), 1e-12)
    f, d = polynomial(s, steps)
    minus, plus = s[:, None] - s[None, :], s[:, None] + s[None, :]
    near = np.abs(minus) < 1e-9
    first = np.where(near, d[:, None], (f[:, None] - f[None, :]) / np.where(near, 1.0, minus))
    second = (f[:, None] + f[None, :]) / plus
    np.fill_diagonal(second, d)
    total = np.sum(first ** 2 + second ** 2) / 2 + (long_ - len(s)) * np.sum((f / s) ** 2)
    return float(np.sqrt(total / (len(s) * long_)))


def expected_error(update, steps, eps, factor_unit, out_unit):
    """Frobenius error to expect of the result [m, n]: the local errors of
    every step, stretched by the steps after it, and the output's rounding,
    all independent. Factors of the products are off by factor_unit (rms,
    relative), sums of K terms in binary32 by sqrt(K) 2^-24, what is kept of X
    between steps by 2^-23."""
    u = np.asarray(update, np.float64)
    long_ = max(u.shape)
    s = np.linalg.svd(u, compute_uv=False) / (np.sqrt(np.sum(u * u)) + eps)
    kept = 2.0 ** -23
    total = (amplification(s, long_, steps) * 2 * kept * np.linalg.norm(s)) ** 2
    for k in range(steps):
        x, top = np.linalg.norm(s), s.max()
        gram, square = np.linalg.norm(s ** 2), top ** 2
        poly = np.linalg.norm(B * s ** 2 + C * s ** 4)
        slope = np.abs(B + 2 * C * s ** 2).max()
        d_gram = (2 * factor_unit + np.sqrt(long_) * 2.0 ** -24) * x * top
        d_square = (2 * factor_unit + np.sqrt(len(s)) * 2.0 ** -24) * gram * square
        d_poly = slope * d_gram + C * d_square + factor_unit * poly
        d_next = d_poly * top + (2 * factor_unit + np.sqrt(len(s)) * 2.0 ** -24) * poly * top + kept * (A * x + poly * top)
        s = polynomial(s, 1)[0]
        total += (amplification(np.abs(s), long_, steps - k - 1) * d_next) ** 2
    return float(np.sqrt(total + (out_unit / 2 * np.linalg.norm(s)) ** 2))


def float32_error(update, steps, eps):
    """Frobenius error that the iteration makes on [m, n] when X, A and B are
    held in binary32 and every product and sum is rounded to it (the norm and
    X_0's division are exact but for one rounding)."""
    u = np.asarray(update, np.float64)
    x = (u / (np.sqrt(np.sum(u * u)) + eps)).astype(np.float32)
    a, b, c = np.float32(A), np.float32(B), np.float32(C)
    for _ in range(steps):
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return float(np.linalg.norm(x.astype(np.float64) - orthogonalize(u, steps, eps)))
