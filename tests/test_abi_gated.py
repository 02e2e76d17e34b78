"""The gated layers reject invalid arguments on the host with the documented
status, before any HIP call (so these run without a GPU)."""

import os

import pytest
import torch

SUCCESS, INVALID, WS_SMALL, HIP, UNSUPPORTED = 0, 1, 2, 3, 4
F = 0x1000   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def dmr():
    import differentiable_mesh_rasterization_amd as pkg

    if not os.path.exists(pkg.LIB_PATH):
        from differentiable_mesh_rasterization_amd import build

        build.build()
    return pkg


def _fwd(dmr, x=F, R=10, cin=8, off=F, N=2, w=F, b=None, cout=4, act=0, dtype=0, y=F):
    return dmr.lib().dmr_grouped_gated_linear_fwd(x, R, cin, off, N, w, b, cout, act, dtype, y, None)


def _bwd(dmr, x=F, R=10, cin=8, off=F, N=2, w=F, b=None, cout=4, act=0, dtype=0, g=F, gx=F, gw=F, gb=F, ws=F, ws_bytes=0):
    return dmr.lib().dmr_grouped_gated_linear_bwd(x, R, cin, off, N, w, b, cout, act, dtype, g, gx, gw, gb, ws, ws_bytes, None)


COMMON = [
    (dict(R=-1), INVALID), (dict(N=-1), INVALID), (dict(N=0), INVALID), (dict(cin=0), INVALID), (dict(cout=0), INVALID),
    (dict(cin=-8), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(off=None), INVALID),
    (dict(act=-1), INVALID), (dict(act=4), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(cin=(1 << 20) + 1), UNSUPPORTED), (dict(cout=(1 << 19) + 1), UNSUPPORTED), (dict(cout=(1 << 31) - 1), UNSUPPORTED),
    (dict(R=1 << 60), UNSUPPORTED), (dict(R=1 << 40), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED),
    (dict(N=1 << 20, cin=1 << 15), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(y=None), INVALID)])
def test_gated_forward_rejects_invalid_arguments(dmr, kw, status):
    assert _fwd(dmr, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(g=None), INVALID), (dict(ws=None), WS_SMALL), (dict(ws_bytes=64), WS_SMALL), (dict(ws=0x1004, ws_bytes=1 << 30), INVALID),
    (dict(gw=None, gb=None), WS_SMALL),
])
def test_gated_backward_rejects_invalid_arguments(dmr, kw, status):
    assert _bwd(dmr, **kw) == status


def test_gated_layer_with_nothing_to_do_is_a_no_op(dmr):
    assert _fwd(dmr, R=0, x=None, w=None, y=None) == SUCCESS
    assert _fwd(dmr, R=0, N=0, off=None, x=None, w=None, y=None) == SUCCESS
    assert _bwd(dmr, R=0, N=0, off=None, x=None, w=None, g=None) == SUCCESS
    assert _bwd(dmr, gx=None, gw=None, gb=None, ws=None) == SUCCESS
    assert _bwd(dmr, R=0, x=None, w=None, g=None, gw=None, gb=None, ws=None) == SUCCESS


def test_gated_workspace_sizes(dmr):
    size, linear = dmr.dmr_grouped_gated_linear_workspace_size, dmr.dmr_grouped_linear_workspace_size
    # the gradients of both products for every row, and the sums of a linear layer of twice the outputs
    for R, N, cin, cout, dtype, each in ((1000, 3, 72, 40, torch.bfloat16, 2), (50000, 3, 37, 129, torch.float32, 4)):
        assert size(R, N, cin, cout, dtype) >= R * 2 * cout * each + linear(R, N, cin, 2 * cout, dtype)
    # narrow layers: sums of pieces alone, a group of r > 128 rows has at most 2 r / 128
    assert 0 < size(100, 3, 64, 128, torch.float32) <= 512
    assert 2 * (2 * 64 * 65) * 4 <= size(1 << 20, 4, 64, 64, torch.bfloat16) < (1 << 20) * 2 * 64 * 2
    assert size(-1, 2, 8, 4, torch.float32) == 0 and size(10, 2, 8, 4, torch.float64) == 0
    assert size(10, 2, 8, 1 << 20, torch.float32) == 0


# groups whose backward pass takes a workgroup of 512 each; whose pieces are
# added by several of 256 each; and, of wider layers, as a linear layer's
@pytest.mark.parametrize("R,N,cin,cout,dtype,fewer", [(100, 1 << 23, 1, 100, torch.float32, (1 << 23) - 8),
                                                      (1000, 1 << 21, 64, 64, torch.float32, 1 << 18),
                                                      (1 << 29, 1 << 21, 512, 256, torch.bfloat16, 1 << 17)])
def test_gated_sums_past_a_launch_are_refused(dmr, R, N, cin, cout, dtype, fewer):
    size, code = dmr.dmr_grouped_gated_linear_workspace_size, dmr.DTYPES[dtype]
    assert size(R, N, cin, cout, dtype) == 0 and size(R, fewer, cin, cout, dtype) > 0
    assert _bwd(dmr, R=R, cin=cin, N=N, cout=cout, dtype=code, ws_bytes=1 << 62) == UNSUPPORTED
    assert _bwd(dmr, R=R, cin=cin, N=fewer, cout=cout, dtype=code, ws_bytes=16) == WS_SMALL


def test_gated_arguments_are_checked_before_the_library(dmr):
    x, off, w = torch.zeros((4, 8)), torch.tensor([0, 1, 4]), torch.zeros((2, 2, 3, 8))
    for kind in ("relu", None, 0):
        with pytest.raises(ValueError):
            dmr.grouped_gated_linear(x, off, w, activation=kind)
    with pytest.raises(ValueError):
        dmr.grouped_gated_linear(x, off, torch.zeros((2, 3, 3, 8)))
    with pytest.raises(ValueError):
        dmr.grouped_gated_linear(x, off, torch.zeros((2, 6, 8)))
    with pytest.raises(ValueError):                 # no GPU tensors
        dmr.grouped_gated_linear(x, off, w)
