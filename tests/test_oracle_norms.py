"""Pins of the oracle of layer norms and of clipped gradients: hand-worked
rows, differences, invariants, and mistakes planted in it that the bounds must
not let pass."""

import numpy as np
import pytest

from oracle import norms


def _case(seed=0, sizes=(3, 0, 5, 1), C=7):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(sizes)])
    return (off, rng.normal(size=(off[-1], C)) + 0.5, rng.normal(size=(len(sizes), C)), rng.normal(size=(len(sizes), C)),
            rng.normal(size=(off[-1], C)))


def test_hand_worked_rows():
    # mean 2, variance 1: deviations -1 and 1; gamma 3, beta 10
    y = norms.layer_norm_forward([[1.0, 3.0]], [0, 1], [[3.0, 3.0]], [[10.0, 10.0]], eps=0.0)
    assert np.array_equal(y, [[7.0, 13.0]])
    # mean 0, variance 3, eps 1: s = 1/2
    assert np.array_equal(norms.layer_norm_forward([[-3.0, 1.0, 1.0, 1.0]], [0, 1], eps=1.0), [[-1.5, 0.5, 0.5, 0.5]])
    # a row of equal values has no gradient but its shift's
    gx, gw, gb = norms.layer_norm_backward([[4.0, 4.0]], [0, 1, 1], None, [[1.0, 2.0]], eps=1.0)
    assert np.array_equal(gx, [[-0.5, 0.5]]) and not gw.any() and np.array_equal(gb, [[1.0, 2.0], [0.0, 0.0]])


def test_rows_are_normalised_and_shifts_and_scales_do_not_matter():
    off, x, _, _, _ = _case()
    y = norms.layer_norm_forward(x, off, eps=0.0)
    assert np.allclose(y.mean(axis=1), 0.0, atol=1e-14) and np.allclose((y * y).mean(axis=1), 1.0)
    assert np.allclose(norms.layer_norm_forward(4.0 * x - 3.0, off, eps=0.0), y)


@pytest.mark.parametrize("weighted", [True, False])
def test_gradients_against_differences(weighted):
    off, x, w, b, g = _case()
    w, b = (w, b) if weighted else (None, None)
    loss = lambda x, w, b: float((norms.layer_norm_forward(x, off, w, b) * g).sum())  # noqa: E731
    grads, h = norms.layer_norm_backward(x, off, w, g), 1e-6
    for k, a in enumerate((x, w, b)):
        if a is None:
            continue
        for i in np.ndindex(a.shape):
            up, down = a.copy(), a.copy()
            up[i] += h
            down[i] -= h
            args = [(x, w, b), (x, w, b)]
            args = [tuple(v if j == k else t for j, t in enumerate((x, w, b))) for v in (up, down)]
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * h) - grads[k][i]) < 1e-7


def test_bounds_hold_binary32_and_refuse_mistakes():
    off, x, w, b, g = _case(1, sizes=(20, 0, 30), C=33)
    x, w, b, g = (t.astype(np.float32).astype(np.float64) for t in (x + 100.0, w, b, g))
    bound = norms.layer_norm_forward_bound(x, off, w, b, "float32")
    ref = norms.layer_norm_forward(x, off, w, b)
    assert (bound < 1e-3).all()
    f = np.float32
    d = (x.astype(f) - x.astype(f).mean(axis=1, dtype=f, keepdims=True))
    d = d - d.mean(axis=1, dtype=f, keepdims=True)
    group = np.searchsorted(off[1:], np.arange(50), side="right")
    y = d / np.sqrt((d * d).mean(axis=1, dtype=f, keepdims=True) + f(1e-5)) * w.astype(f)[group] + b.astype(f)[group]
    assert (np.abs(y - ref) <= bound).all()
    # one value fewer in the variance; eps outside the root; the wrong group
    s = np.sqrt(x.var(axis=1, ddof=1, keepdims=True) + 1e-5)
    assert (np.abs((x - x.mean(axis=1, keepdims=True)) / s * w[group] + b[group] - ref) > bound).any()
    s = np.sqrt(x.var(axis=1, keepdims=True)) + 1e-5
    assert (np.abs((x - x.mean(axis=1, keepdims=True)) / s * w[group] + b[group] - ref) > bound).any()
    assert (np.abs(norms.layer_norm_forward(x, [0, 21, 21, 50], w, b) - ref) > bound).any()
    gx, gw, gb = norms.layer_norm_backward(x, off, w, g)
    bx, bw, bb = norms.layer_norm_backward_bound(x, off, w, g, "float32")
    # without either mean; a row left out of the sums
    h, s = norms._normalised(x, 1e-5)
    q = g * w[group]
    assert (np.abs(s * (q - h * (q * h).mean(axis=1, keepdims=True)) - gx) > bx).any()
    assert (np.abs(s * (q - q.mean(axis=1, keepdims=True)) - gx) > bx).any()
    g[7] = 0.0
    _, gw2, gb2 = norms.layer_norm_backward(x, off, w, g)
    assert (np.abs(gw2 - gw) > bw).any() and (np.abs(gb2 - gb) > bb).any()


def test_clipping():
    out, n = norms.clip_grad_norm([[3.0], [[4.0]]], 1.0, eps=0.0)
    assert n == [5.0] and np.allclose(out[0], 0.6) and np.allclose(out[1], [[0.8]])
    out, n = norms.clip_grad_norm([[[3.0, 4.0], [0.3, 0.4], [0.0, 0.0]]], 1.0, groups=3, eps=0.0)
    assert np.allclose(n, [5.0, 0.5, 0.0]) and np.allclose(out[0], [[0.6, 0.8], [0.3, 0.4], [0.0, 0.0]])
    out, n = norms.clip_grad_norm([[1.0, np.inf]], 1.0)
    assert n == [np.inf] and out[0][0] == 0.0 and np.isnan(out[0][1])
    assert np.isnan(norms.clip_grad_norm([[1.0, np.nan]], 1.0)[0][0]).all()
