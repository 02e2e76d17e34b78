"""The activations of the gated layers and their derivatives, each alone: one
input of 1 and weights that are the arguments, so that a is exact, and u = 1.

Tolerances: oracle/grouped_gated.py (activation_error) and the rounding to the
type; the derivative comes out as the gradient of the gate's weight."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_gated import _backward, _check, _typed
from oracle.grouped_gated import ACTIVATIONS, HELD, activate, activation_error
from oracle.grouped_linear import TINY, UNIT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _arguments(count):
    rng = np.random.default_rng(0)
    return np.concatenate([np.linspace(-30, 30, count // 2), rng.normal(size=count // 4), 40 * rng.normal(size=count // 8),
                           rng.normal(size=count - count // 2 - count // 4 - count // 8) * 1e-3])


# both forms of the backward pass: 100 hidden values at a time, and all at once
@pytest.mark.parametrize("dtype", list(UNIT))
@pytest.mark.parametrize("act", ACTIVATIONS)
@pytest.mark.parametrize("cout", [100, 4000])
def test_activations_keep_the_digits_of_both_tails(dmr, act, cout, dtype):
    say(f"[gpu] {act} alone, {dtype}, {cout} at a time")
    N = 4000 // cout
    a, a64 = _typed(_arguments(4000).reshape(N, cout, 1), dtype)
    w = torch.stack([a, torch.ones_like(a)], dim=1)
    x, off = torch.ones((N, 1), dtype=a.dtype, device=DEV), torch.arange(N + 1, device=DEV)
    y = dmr.grouped_gated_linear(x, off, w, None, act)
    _, gw, _ = _backward(dmr, x, off, w, None, torch.ones_like(y), act)
    (value, slope, _), errors = activate(a64[..., 0], act), activation_error(a64[..., 0], act)
    for got, ref, own, held, what in ((y, value, errors[0], 0.0, "y"), (gw[:, 0, :, 0], slope, errors[1], HELD[dtype], "slope"),
                                      (gw[:, 1, :, 0], value, errors[0], HELD[dtype], "value")):
        e = own + held * (np.abs(ref) + own)
        _check(got, ref, e + UNIT[dtype] * (np.abs(ref) + e) + TINY[dtype], what)
