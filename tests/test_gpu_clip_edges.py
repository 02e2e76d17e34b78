"""Clipping at the edges of its limits.

Tolerances: as in test_gpu_norms.py (oracle/norms.py)."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_norms import _check, _typed
from oracle.norms import clip_bound, clip_grad_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", [50, 70000])       # one workgroup for a group, and chunks
def test_clip_of_zeros_to_zero_without_eps(dmr, size, dtype):
    # 0 / 0: nothing to scale; other groups are scaled to zero
    say(f"[gpu] clip of zeros to 0, {size} {dtype}")
    g = torch.zeros((3, size), dtype=dtype, device=DEV)
    g[1] = 1.0
    (out,), n = dmr.clip_grad_norm([g], 0.0, groups=3, eps=0.0)
    assert (out == 0).all() and n[0] == 0 and n[1] > 0 and n[2] == 0
    (out,), n = dmr.clip_grad_norm([g[0]], 0.0, eps=0.0)
    assert (out == 0).all() and (n == 0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size", [50, 70000])
@pytest.mark.parametrize("scale,max_norm", [(1e30, 1e-12), (1e36, 1e-10), (3e37, 1e-40), (1e20, 1e-44), (1e5, 1e-37)])
def test_clip_by_factors_below_the_normal_range(dmr, scale, max_norm, size, dtype):
    # max_norm / norm is 1e-42 to 1e-77, the clipped values are not that small
    say(f"[gpu] clip of {size} {dtype} of {scale} to {max_norm}")
    g, g64 = _typed(scale * np.random.default_rng(0).normal(size=(2, size)), dtype)
    limit = float(np.float32(max_norm))
    (out,), n = dmr.clip_grad_norm([g], limit, groups=2)
    (ref,), _ = clip_grad_norm([g64], limit, 2)
    _check(out, ref, clip_bound(ref, dtype), "clipped")
