"""The per-group linear layers and the orthogonalised updates reject invalid
arguments on the host with the documented status, before any HIP call (so
these run without a GPU)."""

import ctypes
import os

import pytest

SUCCESS, INVALID, WS_SMALL, HIP, UNSUPPORTED = 0, 1, 2, 3, 4
P = ctypes.c_void_p
F = 0x1000   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def dmr():
    import differentiable_mesh_rasterization_amd as pkg

    if not os.path.exists(pkg.LIB_PATH):
        from differentiable_mesh_rasterization_amd import build

        build.build()
    return pkg


def _fwd(dmr, x=F, R=10, cin=8, off=F, N=2, w=F, b=None, cout=4, dtype=0, y=F):
    return dmr.lib().dmr_grouped_linear_fwd(P(x), R, cin, P(off), N, P(w), P(b), cout, dtype, P(y), None)


def _bwd(dmr, x=F, R=10, cin=8, off=F, N=2, w=F, cout=4, dtype=0, g=F, gx=F, gw=F, gb=F, ws=F, ws_bytes=0):
    return dmr.lib().dmr_grouped_linear_bwd(P(x), R, cin, P(off), N, P(w), cout, dtype, P(g), P(gx), P(gw), P(gb), P(ws),
                                            ws_bytes, None)


COMMON = [
    (dict(R=-1), INVALID), (dict(N=-1), INVALID), (dict(N=0), INVALID), (dict(cin=0), INVALID), (dict(cout=0), INVALID),
    (dict(cin=-8), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(off=None), INVALID),
    (dict(cin=(1 << 20) + 1), UNSUPPORTED), (dict(cout=1 << 21), UNSUPPORTED), (dict(R=1 << 60), UNSUPPORTED),
    (dict(R=1 << 40), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED), (dict(N=1 << 20, cin=1 << 15), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID)])
def test_layer_forward_rejects_invalid_arguments(dmr, kw, status):
    assert _fwd(dmr, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(g=None), INVALID),
    (dict(x=None, gx=None, gb=None), INVALID), (dict(w=None, gw=None, gb=None), INVALID),
    (dict(ws=None), WS_SMALL), (dict(ws_bytes=64), WS_SMALL), (dict(ws=0x1004, ws_bytes=1 << 30), INVALID),
])
def test_layer_backward_rejects_invalid_arguments(dmr, kw, status):
    assert _bwd(dmr, **kw) == status


def test_layer_with_nothing_to_do_is_a_no_op(dmr):
    assert _fwd(dmr, R=0, x=None, w=None, y=None) == SUCCESS
    assert _fwd(dmr, R=0, N=0, off=None, x=None, w=None, y=None) == SUCCESS
    assert _bwd(dmr, R=0, N=0, off=None, x=None, w=None, g=None) == SUCCESS
    assert _bwd(dmr, gx=None, gw=None, gb=None, ws=None) == SUCCESS


def test_layer_workspace_sizes(dmr):
    import torch

    size = dmr.dmr_grouped_linear_workspace_size
    assert 0 < size(10, 2, 8, 4, torch.float32) <= 512          # one piece a group: no partial results
    # a group of r > rows rows has at most 2 r / rows pieces of (in + 1) out values
    big = size(1 << 20, 4, 64, 64, torch.bfloat16)
    assert big >= 2 * (64 * 64 + 64) * 4
    assert size(-1, 2, 8, 4, torch.float32) == 0 and size(10, 2, 8, 4, torch.float64) == 0


def _orth(dmr, u=F, B=2, m=8, n=8, dtype=0, steps=5, eps=1e-7, out=F, ws=F, ws_bytes=1 << 20):
    return dmr.lib().dmr_orthogonalize(P(u), B, m, n, dtype, steps, eps, P(out), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(m=0), INVALID), (dict(n=-3), INVALID), (dict(dtype=7), INVALID), (dict(u=None), INVALID),
    (dict(out=None), INVALID), (dict(steps=0), INVALID), (dict(steps=-1), INVALID), (dict(steps=65), UNSUPPORTED),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(m=1 << 21), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED), (dict(B=1 << 26, m=512, n=512), UNSUPPORTED),
    (dict(ws=None), WS_SMALL), (dict(m=512, n=512, ws_bytes=4096), WS_SMALL), (dict(ws=0x1008), INVALID),
])
def test_update_rejects_invalid_arguments(dmr, kw, status):
    assert _orth(dmr, **kw) == status


def test_update_of_no_matrix_is_a_no_op(dmr):
    assert _orth(dmr, B=0, u=None, out=None, ws=None, ws_bytes=0) == SUCCESS


def test_update_workspace_sizes(dmr):
    import torch

    size = dmr.dmr_orthogonalize_workspace_size
    assert size(4, 16, 16, torch.float32) > 0
    assert size(1, 512, 512, torch.float32) > 512 * 512 * 4 * 2
    assert size(1, 512, 512, torch.bfloat16) <= size(1, 512, 512, torch.float32)
    assert size(2, 512, 512, torch.float32) > size(1, 512, 512, torch.float32)
    assert size(0, 5, 5, torch.float32) > 0
    assert size(1, 0, 5, torch.float32) == 0 and size(1, 5, 5, torch.int64) == 0
