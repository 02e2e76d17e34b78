"""How tight the bounds of the gated layers are: mistakes of the size of one
rounding more than the definition has, planted in the oracle, must be refused."""

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
