"""Sizes whose launches would pass 2^32 - 1 work-items (what HIP takes in one
launch) are refused as unsupported, before any HIP call (so these run without a
GPU), and the largest ones below that are not."""

import ctypes
import os

import pytest
import torch

INVALID, WS_SMALL, UNSUPPORTED = 1, 2, 4
P = ctypes.c_void_p
F = 0x1000   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def dmr():
    import differentiable_mesh_rasterization_amd as pkg

    if not os.path.exists(pkg.LIB_PATH):
        from differentiable_mesh_rasterization_amd import build

        build.build()
    return pkg


# matrices of one workgroup of 256 and of 1024 threads; of 64 workgroups of 256
# (their norm); of many 64 x 64 tiles of 512
@pytest.mark.parametrize("B,m,n", [(1 << 24, 3, 3), (1 << 22, 33, 33), (1 << 18, 65, 65), (1 << 15, 1024, 1024), (8, 65536, 65536)])
def test_updates_past_a_launch_are_refused(dmr, B, m, n):
    assert dmr.dmr_orthogonalize_workspace_size(B, m, n, torch.float32) == 0
    assert dmr.lib().dmr_orthogonalize(P(F), B, m, n, 0, 5, 1e-7, P(F), P(F), 1 << 62, None) == UNSUPPORTED
    assert dmr.dmr_orthogonalize_workspace_size(B - B // 16 - 1 if B > 16 else B - 1, m, n, torch.float32) > 0
