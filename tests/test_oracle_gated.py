"""Pins of the oracle of the gated layers: hand-worked values, differences, and
mistakes planted in it that the bounds must not let pass."""

import math

import numpy as np
import pytest

from oracle import grouped_gated as gated

KINDS = list(gated.ACTIVATIONS)


def _case(seed=0, sizes=(3, 0, 5, 1), C=4, F=3):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(sizes)])
    R, N = off[-1], len(sizes)
    return (off, rng.normal(size=(R, C)), rng.normal(size=(N, 2, F, C)), rng.normal(size=(N, 2, F)), rng.normal(size=(R, F)))


def test_hand_worked_values():
    # one row, C = 1, F = 1: a = 2 x + 1 = 3, u = -x = -1
    x, w, b = [[1.0]], [[[[2.0]], [[-1.0]]]], [[[1.0], [0.0]]]
    want = {"silu": -3 / (1 + math.exp(-3)), "sigmoid": -1 / (1 + math.exp(-3)), "gelu": -3 * 0.9986501019683699,
            "gelu_tanh": -1.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * (3 + 0.044715 * 27)))}
    for kind in KINDS:
        assert np.allclose(gated.gated_forward(x, [0, 1], w, b, kind), want[kind], rtol=1e-14)
    # the two planes are not exchangeable
    assert not np.allclose(gated.gated_forward(x, [0, 1], np.asarray(w)[:, ::-1], np.asarray(b)[:, ::-1]), want["silu"])


@pytest.mark.parametrize("kind", KINDS)
def test_activations(kind):
    a = np.array([-40.0, -5.0, -1.0, -1e-3, 0.0, 1e-3, 0.7, 5.0, 40.0])
    value, slope, _ = gated.activate(a, kind)
    h = 1e-5
    assert np.allclose((gated.activate(a + h, kind)[0] - gated.activate(a - h, kind)[0]) / (2 * h), slope, atol=1e-9)
    # the bounds' constants on the derivatives
    fine = np.linspace(-12, 12, 24001)
    s = gated.activate(fine, kind)[1]
    assert np.abs(s).max() <= 1.13 and np.abs(np.diff(s)).max() <= 1e-3 * 1.0
    assert abs(value[-1] - (1.0 if kind == "sigmoid" else 40.0)) < 1e-12 and abs(value[0]) < 1e-15


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("biased", [True, False])
def test_gradients_against_differences(kind, biased):
    off, x, w, b, g = _case()
    b = b if biased else None
    grads, h = gated.gated_backward(x, off, w, b, g, kind), 1e-6
    for k, t in enumerate((x, w, b)):
        if t is None:
            continue
        for i in np.ndindex(t.shape):
            moved = []
            for d in (h, -h):
                v = t.copy()
                v[i] += d
                args = [v if j == k else s for j, s in enumerate((x, w, b))]
                moved.append((gated.gated_forward(args[0], off, args[1], args[2], kind) * g).sum())
            assert abs((moved[0] - moved[1]) / (2 * h) - grads[k][i]) < 1e-7


@pytest.mark.parametrize("kind", KINDS)
def test_bounds_refuse_mistakes(kind):
    off, x, w, b, g = _case(1, (40, 0, 30), 16, 8)
    y, bound = gated.gated_forward(x, off, w, b, kind), gated.gated_forward_bound(x, off, w, b, "bfloat16", kind)
    assert (bound < 0.02 * np.abs(y) + 0.02).all()
    grads, bounds = gated.gated_backward(x, off, w, b, g, kind), gated.gated_backward_bound(x, off, w, b, g, "bfloat16", kind)

    def caught(args, name=kind):
        x2, off2, w2, b2, g2 = args
        wrong = gated.gated_backward(x2, off2, w2, b2, g2, name)
        return (np.abs(gated.gated_forward(x2, off2, w2, b2, name) - y) > bound).any(), [
            (np.abs(v - r) > e).any() for v, r, e in zip(wrong, grads, bounds)]

    forward, backward = caught((x, off, w[:, ::-1], b[:, ::-1], g))       # the planes exchanged
    assert forward and all(backward)
    forward, backward = caught((x, [0, 41, 41, 70], w, b, g))             # a row of the wrong group
    assert forward and all(backward)
    forward, backward = caught((x, off, w, None, g))                      # no bias
    assert forward and all(backward)
    g2 = g.copy()
    g2[5] = 0
    assert all(caught((x, off, w, b, g2))[1])                             # a row left out
    other = {"gelu": "silu", "silu": "gelu", "gelu_tanh": "silu", "sigmoid": "silu"}[kind]
    forward, backward = caught((x, off, w, b, g), other)
    assert forward and all(backward)
    # in float32 the two forms of gelu are told apart
    if kind.startswith("gelu"):
        other = "gelu" if kind == "gelu_tanh" else "gelu_tanh"
        assert (np.abs(gated.gated_forward(x, off, w, b, other) - y) > gated.gated_forward_bound(x, off, w, b, "float32", kind)).any()
