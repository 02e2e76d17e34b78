"""The example that fits one decoder per mesh through the rasterizer: layers,
projection, rasterization and orthogonalised updates run together, and the
depth error falls."""

import importlib.util
import os

import numpy as np
import pytest

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


def test_decoders_learn_the_target_shapes():
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fit_decoders.py")
    spec = importlib.util.spec_from_file_location("fit_decoders", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    say("[gpu] fit 4 decoders, 40 steps")
    losses = example.fit(steps=40)
    assert np.isfinite(losses).all()
    # the shapes' depth differs by 0.2 at most: the start is below 0.2^2, and
    # the decoders, which can represent the target well, take most of it away
    assert 1e-4 < losses[0] < 0.04
    assert losses[-1] < 0.25 * losses[0]
