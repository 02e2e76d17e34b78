"""Sizes whose launches would pass 2^32 - 1 work-items (what HIP takes in one
launch) are refused as unsupported, before any HIP call (so these run without a
GPU), and the largest ones below that are not."""

import ctypes
import os

import pytest
import torch

WS_SMALL, UNSUPPORTED = 2, 4
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


# groups whose weights' gradients take a workgroup of 256 each, 16 each, and
# whose pieces are added by 17 workgroups of 256 each; and fewer of them
@pytest.mark.parametrize("R,N,cin,cout,dtype,fewer", [(10, 1 << 24, 1, 1, torch.float32, (1 << 24) - 64),
                                                      (1 << 29, 1 << 21, 512, 512, torch.bfloat16, 1 << 17),
                                                      (1 << 21, 1 << 20, 64, 64, torch.float32, 1 << 19)])
def test_sums_over_rows_past_a_launch_are_refused(dmr, R, N, cin, cout, dtype, fewer):
    size, code = dmr.dmr_grouped_linear_workspace_size, dmr.DTYPES[dtype]
    backward = dmr.lib().dmr_grouped_linear_bwd
    assert size(R, N, cin, cout, dtype) == 0
    for gx, gw, gb in ((F, F, F), (None, F, None), (None, None, F)):
        assert backward(P(F), R, cin, P(F), N, P(F), cout, code, P(F), P(gx), P(gw), P(gb), P(F), 1 << 62, None) == UNSUPPORTED
    assert size(R, fewer, cin, cout, dtype) > 0


def test_rows_of_as_many_groups_are_not_refused(dmr):
    # the rows' gradient walks its tiles, whatever their number: only the workspace of the sums is missing
    backward = dmr.lib().dmr_grouped_linear_bwd
    assert backward(P(F), 10, 1, P(F), (1 << 24) - 64, P(F), 1, 0, P(F), P(F), P(F), None, P(F), 16, None) == WS_SMALL


def test_plans_refuse_what_the_calls_refuse(dmr):
    plan, tile = dmr.dmr_grouped_linear_plan, dmr.dmr_orthogonalize_tile
    assert plan(1 << 20, 4, 64, 64, torch.bfloat16)["y_rows"] == 256
    for bad in ((-1, 2, 8, 4, torch.float32), (10, 0, 8, 4, torch.float32), (10, 2, 0, 4, torch.float32),
                (10, 2, 8, 1 << 21, torch.float32), (10, 2, 8, 4, torch.float64)):
        with pytest.raises(dmr.DmrError):
            plan(*bad)
    assert dmr.lib().dmr_grouped_linear_plan(10, 2, 8, 4, 0, 1, None) == 1
    assert tile(4, 16, 16) == 0 and tile(1, 200, 300) == 64
    assert tile(0, 16, 16) == tile(2, 0, 5) == tile(1 << 40, 200, 300) == -1
