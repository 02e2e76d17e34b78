"""How tight the bounds of the gated layers are: mistakes of the size of one
rounding more than the definition has, planted in the oracle, must be refused."""

import os
import re

import numpy as np
import pytest
import torch

from oracle import grouped_gated as gated

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def _rounded(a, dtype):
    return torch.from_numpy(np.asarray(a, np.float64)).to(TORCH[dtype]).to(torch.float64).numpy()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gradients_rounded_before_their_products_are_refused(dtype):
    rng = np.random.default_rng(0)
    off = np.array([0, 1, 2, 40])
    x, w, g = (_rounded(rng.normal(size=s), dtype) for s in ((40, 8), (3, 2, 6, 8), (40, 6)))
    a, u = gated._projections(x, off, w, None)
    act, slope, _ = gated.activate(a, "silu")
    back = np.stack([g * u * slope, g * act], axis=1)
    ref, bound = gated.gated_backward(x, off, w, None, g), gated.gated_backward_bound(x, off, w, None, g, dtype)
    once = [_rounded(v, dtype) for v in gated._products(x, off, w, back)]
    assert all((np.abs(v - r) <= e).all() for v, r, e in zip(once, ref, bound))
    twice = [_rounded(v, dtype) for v in gated._products(x, off, w, _rounded(back, dtype))]
    # (not of the biases: a single row's gradient is the rounded value itself)
    assert all((np.abs(v - r) > e).any() for v, r, e in zip(twice[:2], ref, bound))
    # as pairs of bfloat16 they pass
    high = _rounded(back, "bfloat16")
    pairs = [_rounded(v, dtype) for v in gated._products(x, off, w, high + _rounded(back - high, "bfloat16"))]
    assert all((np.abs(v - r) <= e).all() for v, r, e in zip(pairs, ref, bound))


@pytest.mark.parametrize("kind", gated.ACTIVATIONS)
def test_derivatives_that_the_bounds_count_with(kind):
    a = np.linspace(-15, 15, 300001)
    slope = gated.activate(a, kind)[1]
    second = np.gradient(slope, a)
    assert np.allclose(gated.curvature(a, kind)[1:-1], second[1:-1], atol=1e-7)
    assert np.abs(second).max() <= 1 and np.abs(np.gradient(second, a)).max() <= 2


@pytest.mark.parametrize("kind", gated.ACTIVATIONS)
def test_activations_that_are_off_in_their_tails_are_refused(kind):
    # by 1e-4 at 10 to 30: below zero the value, above it what it lacks of its limit
    far = np.linspace(10, 30, 41)
    for a in (-far, far):
        value, slope, _ = gated.activate(a, kind)
        own = gated.activation_error(a, kind)
        for ref, e in ((value, own[0]), (slope, own[1])):
            there = np.abs(ref) > 1e-29      # an exponential below 2^-126 may vanish: 1e-4 of these is not that small
            assert (np.abs(1e-4 * ref) > e)[there].all()
    # and through a whole layer of one input, where a may be e = 4 2^-23 |a| off: gelu's tails change by |a| e
    # relatively, and e^2 / 2 is more than they are from about -6 on
    a = np.linspace(-12, -4, 33) if kind in ("silu", "sigmoid") else np.linspace(-4, -2, 33)
    w = np.stack([a, np.ones_like(a)])[None, :, :, None]
    y, bound = gated.gated_forward([[1.0]], [0, 1], w, None, kind), gated.gated_forward_bound([[1.0]], [0, 1], w, None, "float32", kind)
    assert (1e-4 * np.abs(y) > bound).all()


def test_gelus_tail_is_the_normal_distributions():
    # t Q(t) with the coefficients of the kernel, against 1/2 erfcx(a / sqrt(2)): the largest relative
    # error is below half a step of float32 (2^-24)
    scipy = pytest.importorskip("scipy.special")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_mesh_rasterization_amd", "csrc",
                        "grouped_gated.hip")
    with open(path) as f:
        text = re.search(r"constexpr float q\[9\] = \{([^}]*)\}", f.read()).group(1)
    q = [float(np.float32(v.strip().rstrip("f"))) for v in text.split(",")]
    a = np.linspace(0.0, 13.5, 200001)
    t = 1.0 / (1.0 + 0.27 * a)
    fit = t * np.polynomial.polynomial.polyval(t, q)
    off = fit / (0.5 * scipy.erfcx(a / np.sqrt(2.0))) - 1.0
    assert len(q) == 9 and np.abs(off).max() <= 3.6e-8
