"""Every tile that the per-group layers and the orthogonalised updates are
computed by, each asserted to be the one that the call takes: products of
several steps with a remainder, rows, columns and groups that end inside a
tile, empty groups, and weight gradients cut into pieces.

Tolerances: as in test_gpu_operators.py for the layer, as in
test_gpu_update_accuracy.py for the updates."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from oracle.grouped_linear import (backward_error_bound, forward_error_bound, grouped_linear_backward,
                                   grouped_linear_forward)
from test_gpu_update_accuracy import check_update

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
HALF = ["float16", "bfloat16"]
ALL = list(TORCH)


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _typed(rng, shape, dtype):
    """(device tensor of the type, the values it holds in float64)"""
    t = torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(TORCH[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)


def _check(got, ref, bound, what):
    err = np.abs(got.to(torch.float64).cpu().numpy() - ref)
    assert (err <= bound).all(), (what, float((err / bound).max()))   # a NaN fails too


def _plan(dmr, sizes, cin, cout, dtype):
    return dmr.dmr_grouped_linear_plan(sum(sizes), len(sizes), cin, cout, TORCH[dtype])


# (sizes, cin, cout, types, tile: columns and rows); cin of 200: 3 1/8 steps of
# k in 16 bits, 6 1/4 in float32
FORWARD = [([9, 0, 1, 16], 200, 140, ALL, (64, 16)), ([9, 0, 1, 16], 201, 139, ALL, (64, 16)),
           ([900, 0, 130], 200, 12, ALL, (16, 128)), ([900, 0, 130], 203, 3, ALL, (16, 128)),
           ([900, 0, 130], 200, 140, ALL, (64, 128)), ([900, 0, 130], 203, 139, ALL, (64, 128)),
           ([66000, 0, 130], 200, 56, HALF, (64, 256)), ([66000, 0, 130], 203, 51, HALF, (64, 256)),
           ([17000, 0, 130, 1], 200, 136, ALL, (128, 128)), ([17000, 0, 130, 1], 203, 139, ALL, (128, 128)),
           ([28000, 0, 130, 1, 700], 328, 264, HALF, (256, 256)), ([30000, 300], 64, 264, HALF, (256, 256))]


@pytest.mark.parametrize("sizes,cin,cout,dtype,tile", [(s, i, o, d, t) for s, i, o, ds, t in FORWARD for d in ds])
def test_rows_tiles(dmr, sizes, cin, cout, dtype, tile):
    say(f"[gpu] rows {dtype} {cin}->{cout} sizes {sizes} tile {tile}")
    plan = _plan(dmr, sizes, cin, cout, dtype)
    assert (plan["y_columns"], plan["y_rows"]) == tile
    rng, off = np.random.default_rng(cin), _offsets(sizes)
    (x, x64), (w, w64) = _typed(rng, (sum(sizes), cin), dtype), _typed(rng, (len(sizes), cout, cin), dtype)
    b, b64 = _typed(rng, (len(sizes), cout), dtype)
    y = torch.full((x.shape[0], cout), float("nan"), dtype=x.dtype, device=DEV)
    dmr.dmr_grouped_linear_fwd(x, torch.from_numpy(off).to(DEV), w, b, y)
    _check(y, grouped_linear_forward(x64, off, w64, b64), forward_error_bound(x64, off, w64, b64, dtype), "y")


BACKWARD = [([9, 0, 1, 16], 140, 200, ALL, (64, 16)), ([9, 0, 1, 16], 139, 201, ALL, (64, 16)),
            ([900, 0, 130], 12, 200, ALL, (16, 128)), ([900, 0, 130], 3, 203, ALL, (16, 128)),
            ([900, 0, 130], 140, 200, ALL, (64, 128)), ([900, 0, 130], 139, 203, ALL, (64, 128)),
            ([66000, 0, 130], 56, 200, HALF, (64, 256)), ([66000, 0, 130], 51, 203, HALF, (64, 256)),
            ([17000, 0, 130, 1], 136, 200, ALL, (128, 128)), ([17000, 0, 130, 1], 139, 203, ALL, (128, 128)),
            ([14000, 0, 130, 1, 700], 264, 328, HALF, (256, 256)), ([15000, 300], 264, 64, HALF, (256, 256))]


@pytest.mark.parametrize("sizes,cin,cout,dtype,tile", [(s, i, o, d, t) for s, i, o, ds, t in BACKWARD for d in ds])
def test_rows_gradient_tiles(dmr, sizes, cin, cout, dtype, tile):
    say(f"[gpu] rows' gradient {dtype} {cin}->{cout} sizes {sizes} tile {tile}")
    plan = _plan(dmr, sizes, cin, cout, dtype)
    assert (plan["grad_x_columns"], plan["grad_x_rows"]) == tile
    rng, off = np.random.default_rng(cin), _offsets(sizes)
    x, (w, w64) = torch.empty((sum(sizes), cin), dtype=TORCH[dtype], device=DEV), _typed(rng, (len(sizes), cout, cin), dtype)
    g, g64 = _typed(rng, (sum(sizes), cout), dtype)
    gx = torch.full(x.shape, float("nan"), dtype=x.dtype, device=DEV)
    dmr.dmr_grouped_linear_bwd(x, torch.from_numpy(off).to(DEV), w, g, gx, None, None)     # alone
    zeros = np.zeros((sum(sizes), cin))
    _check(gx, grouped_linear_backward(zeros, off, w64, g64)[0], backward_error_bound(zeros, off, w64, g64, dtype)[0], "gx")


# side of the weight gradient's tile; groups of no rows, of one piece and of
# several; weights above and below the 65536 values that the pieces are added
# in two ways for
WEIGHTS = [([900, 0, 130], 56, 40, ALL, 64), ([9000, 0, 1, 130], 64, 60, ALL, 64), ([9000, 0, 1, 130], 61, 63, ALL, 64),
           ([3000, 0, 1, 130], 200, 136, ALL, 128), ([3000, 0, 1, 130], 264, 256, ALL, 128),
           ([3000, 0, 1, 130], 263, 255, ALL, 128), ([100] * 3, 264, 40, ALL, 128),
           ([2500, 0, 1, 130] + [600] * 10 + [513, 77], 264, 328, HALF, 256),
           ([700] * 33, 136, 520, HALF, 256), ([600, 500] * 9, 144, 264, HALF, 128)]


@pytest.mark.parametrize("sizes,cin,cout,dtype,side", [(s, i, o, d, t) for s, i, o, ds, t in WEIGHTS for d in ds])
def test_weight_gradient_tiles(dmr, sizes, cin, cout, dtype, side):
    say(f"[gpu] weights' gradient {dtype} {cin}->{cout} sizes {sizes if len(sizes) < 9 else len(sizes)} side {side}")
    plan = _plan(dmr, sizes, cin, cout, dtype)
    assert plan["grad_weight_side"] == side
    rng, off = np.random.default_rng(cin), _offsets(sizes)
    N = len(sizes)
    (x, x64), (g, g64) = _typed(rng, (sum(sizes), cin), dtype), _typed(rng, (sum(sizes), cout), dtype)
    w, w64 = _typed(rng, (N, cout, cin), dtype)
    ref, bound = grouped_linear_backward(x64, off, w64, g64), backward_error_bound(x64, off, w64, g64, dtype)
    ws = torch.empty(dmr.dmr_grouped_linear_workspace_size(sum(sizes), N, cin, cout, x.dtype), dtype=torch.uint8, device=DEV)
    for rows_too in (False, True):     # the weights' gradients alone, then with the rows'
        out = [torch.full(s, float("nan"), dtype=x.dtype, device=DEV) for s in (x.shape, w.shape, (N, cout))]
        if not rows_too:
            out[0] = None
        dmr.dmr_grouped_linear_bwd(x, torch.from_numpy(off).to(DEV), w, g, *out, ws)
        for v, r, b, what in zip(out, ref, bound, ("gx", "gw", "gb")):
            if v is not None:
                _check(v, r, b, what)


def test_cut_weight_gradients_are_among_them(dmr):
    cut = {(_plan(dmr, s, i, o, d)["grad_weight_side"], i * o + o > 65536)
           for s, i, o, ds, _ in WEIGHTS for d in ds if max(s) > _plan(dmr, s, i, o, d)["piece_rows"] and sum(s) > 1024}
    assert {(64, False), (128, False), (128, True), (256, True)} <= cut
    together = {_plan(dmr, s, i, o, d)["together"] for s, i, o, ds, _ in WEIGHTS + BACKWARD for d in ds}
    assert together == {0, 1}


# batches that fill the device with larger tiles: whole ones, and sides that
# end inside them (300 x 420 and 440 x 700 pad to 320 x 448 and 448 x 704)
UPDATES = [(2, 300, 420, 64), (22, 300, 420, 128), (22, 420, 300, 128), (16, 512, 512, 128), (9, 640, 700, 128),
           (38, 440, 700, 256), (38, 700, 440, 256), (14, 1024, 1024, 256), (4, 600, 3900, 128)]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("B,m,n,side", UPDATES)
def test_update_tiles(dmr, B, m, n, side, dtype):
    say(f"[gpu] update {dtype} {B} x {m} x {n} side {side}")
    assert dmr.dmr_orthogonalize_tile(B, m, n) == side
    rng = np.random.default_rng(m)
    u, u64 = _typed(rng, (B, m, n), dtype)
    some = sorted({0, B // 2, B - 1})
    # one of them far below eps, one of few strong directions
    u64[some[-1]] *= 1e-9
    if B > 2:
        u64[some[1]] = rng.normal(size=(m, 20)) @ rng.normal(size=(20, n)) + 1e-2 * u64[some[1]]
    u = torch.from_numpy(u64).to(TORCH[dtype])
    u64 = u.to(torch.float64).numpy()
    u = u.to(DEV)
    got = dmr.orthogonalize(u)
    check_update(got[some], u64[some], dtype)
    assert torch.isfinite(got).all()
    assert torch.equal(got, dmr.orthogonalize(u))
    if m == n:     # the iteration of the transpose is the transpose's
        turned = dmr.orthogonalize(u.transpose(1, 2).contiguous()).transpose(1, 2).contiguous()
        check_update(turned[some], u64[some], dtype)
