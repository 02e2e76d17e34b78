"""The layer norms and the clipping of gradients reject invalid arguments on
the host with the documented status, before any HIP call (so these run without
a GPU)."""

import ctypes
import os
import struct

import pytest
import torch

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


def _fwd(dmr, x=F, R=10, C=8, off=F, N=2, w=F, b=F, eps=1e-5, dtype=0, y=F):
    return dmr.lib().dmr_grouped_layer_norm_fwd(x, R, C, off, N, w, b, eps, dtype, y, None)


def _bwd(dmr, x=F, R=10, C=8, off=F, N=2, w=F, eps=1e-5, dtype=0, g=F, gx=F, gw=F, gb=F, ws=F, ws_bytes=0):
    return dmr.lib().dmr_grouped_layer_norm_bwd(x, R, C, off, N, w, eps, dtype, g, gx, gw, gb, ws, ws_bytes, None)


COMMON = [
    (dict(R=-1), INVALID), (dict(N=-1), INVALID), (dict(N=0), INVALID), (dict(C=0), INVALID), (dict(C=-8), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(off=None), INVALID), (dict(x=None), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(C=(1 << 20) + 1), UNSUPPORTED), (dict(R=1 << 60), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED),
    (dict(N=1 << 20, C=1 << 15), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(y=None), INVALID)])
def test_layer_norm_forward_rejects_invalid_arguments(dmr, kw, status):
    assert _fwd(dmr, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(g=None), INVALID), (dict(ws=None), WS_SMALL), (dict(ws_bytes=64), WS_SMALL),
    (dict(ws=0x1004, ws_bytes=1 << 30), INVALID), (dict(gx=None, gb=None), WS_SMALL), (dict(gx=None, gw=None), WS_SMALL),
])
def test_layer_norm_backward_rejects_invalid_arguments(dmr, kw, status):
    assert _bwd(dmr, **kw) == status


def test_layer_norm_with_nothing_to_do_is_a_no_op(dmr):
    assert _fwd(dmr, R=0, x=None, w=None, b=None, y=None) == SUCCESS
    assert _fwd(dmr, R=0, N=0, off=None, x=None, y=None) == SUCCESS
    assert _bwd(dmr, R=0, N=0, off=None, x=None, g=None) == SUCCESS
    assert _bwd(dmr, gx=None, gw=None, gb=None, ws=None) == SUCCESS
    assert _bwd(dmr, R=0, x=None, g=None, gw=None, gb=None, ws=None) == SUCCESS


def test_layer_norm_workspace_sizes(dmr):
    size = dmr.dmr_grouped_layer_norm_workspace_size
    assert size(10, 2, 8, torch.float32) > 0
    # two slots of 2 C sums a workgroup, of at most 2048
    assert 4 * 2048 * 64 * 4 <= size(1 << 20, 4, 64, torch.bfloat16) <= 4 * 2048 * 64 * 4 + 1024
    # rows too long for registers: their statistics beside slots for fewer workgroups
    assert 16 * 100 <= size(100, 4, 1 << 20, torch.float32) < 1 << 26
    assert size(-1, 2, 8, torch.float32) == 0 and size(10, 2, 8, torch.float64) == 0 and size(10, 0, 8, torch.float32) == 0


def _clip(dmr, spans=((F, F, 10, 0), (F + 64, F + 64, 3, 2)), groups=2, max_norm=1.0, eps=1e-6, norms=F, ws=F, ws_bytes=1 << 20,
          count=None, table=True):
    packed = struct.pack("QQqii" * len(spans), *[v for s in spans for v in (*s, 0)]) if table else None
    return dmr.lib().dmr_clip_norm(packed, len(spans) if count is None else count, groups, max_norm, eps, norms, ws, ws_bytes,
                                   None)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=-1), INVALID), (dict(count=-1), INVALID), (dict(table=False), INVALID), (dict(norms=None), INVALID),
    (dict(max_norm=-1.0), INVALID), (dict(max_norm=float("nan")), INVALID), (dict(max_norm=float("inf")), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(spans=((F, F, -1, 0),)), INVALID), (dict(spans=((F, F, 10, 3),)), INVALID), (dict(spans=((0, F, 10, 0),)), INVALID),
    (dict(spans=((F, 0, 10, 0),)), INVALID), (dict(spans=((F, F, 1 << 61, 0),)), UNSUPPORTED),
    (dict(spans=((F, F, 1 << 40, 0),) * 4, groups=1 << 22), UNSUPPORTED), (dict(groups=1 << 31), UNSUPPORTED),
    (dict(spans=((F, F, 1 << 20, 0),), ws=None), WS_SMALL), (dict(spans=((F, F, 1 << 20, 0),), ws_bytes=16), WS_SMALL),
    (dict(spans=((F, F, 1 << 20, 0),), ws=0x1008), INVALID),
])
def test_clipping_rejects_invalid_arguments(dmr, kw, status):
    assert _clip(dmr, **kw) == status


def test_clipping_of_no_group_is_a_no_op(dmr):
    assert _clip(dmr, groups=0, norms=None, ws=None, ws_bytes=0) == SUCCESS


def test_clipping_workspace_sizes(dmr):
    size = dmr.dmr_clip_norm_workspace_size
    small, large = torch.zeros((4, 10)), torch.zeros((4, 1 << 20))
    assert 0 < size([small, small], 4) <= 512       # a workgroup a group: no partial sums
    assert size([large, small], 4) >= 4 * 2 * 8
    with pytest.raises(ValueError):
        size([small], 3)
    with pytest.raises(ValueError):
        size([], 3)
    with pytest.raises(TypeError):
        size([small.double()], 4)


def test_clipping_refuses_outputs_that_share_memory(dmr):
    buf = torch.zeros(40)
    a, b = buf[:10], buf[10:20]
    check = dmr._check_overlap
    check([a, b], [a, b])                                # in place
    check([a, b], [buf[20:30], buf[30:40]])              # elsewhere
    check([a, a], [buf[20:30], buf[30:40]])              # the same input twice
    check([a, b], [a, buf[20:30]])
    for tensors, outs in (([a, a], [a, a]), ([a, b], [b, a]), ([a, b], [buf[20:30], buf[25:35]]), ([a], [buf[5:15]]),
                          ([a, a], [a, buf[20:30]]), ([buf[:20], b], [buf[20:40], b])):
        with pytest.raises(ValueError):
            check(tensors, outs)
