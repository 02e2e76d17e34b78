"""Clipping at the edges of its limits.

Tolerances: as in test_gpu_norms.py (oracle/norms.py)."""

import pytest
import torch

from gpu_util import DEV, require_gpu, say

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
