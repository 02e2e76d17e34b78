"""Every tile that the gated layers are computed by, each asserted to be the
one that the call takes: products of several steps with a remainder and of one
and two steps, rows, columns and groups that end inside a tile, empty groups,
more tiles than the device holds workgroups; and the backward pass in one
kernel, of short and long pieces.

Tolerances: as in test_gpu_gated.py (oracle/grouped_gated.py)."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_gated import _backward, _check, _inputs
from oracle.grouped_gated import gated_backward, gated_backward_bound, gated_forward, gated_forward_bound

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
HALF = ["float16", "bfloat16"]
ALL = list(TORCH)


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


# (sizes, cin, cout, types, tile: columns and rows); cin of 200: 3 1/8 steps of
# k in 16 bits, 6 1/4 in float32
TILES = [([9, 0, 1, 16], 200, 140, ALL, (64, 16)), ([9, 0, 1, 16], 201, 139, ALL, (64, 16)),
         ([900, 0, 130], 200, 140, ALL, (64, 16)), ([900, 0, 130], 203, 139, ALL, (64, 16)),
         ([16300, 0, 130], 200, 12, ALL, (16, 128)), ([16300, 0, 130], 203, 3, ALL, (16, 128)),
         ([3300, 0, 130], 200, 140, ALL, (32, 128)), ([3300, 0, 130], 203, 139, ALL, (32, 128)),
         ([3300, 0, 130], 64, 140, ALL, (32, 128)), ([3300, 0, 130], 100, 140, ALL, (32, 128)),
         ([12000, 0, 130, 1], 200, 136, ALL, (64, 128)), ([12000, 0, 130, 1], 203, 139, ALL, (64, 128)),
         # 258 tiles of rows and three of columns for 256 workgroups; steps of k: 4, 1, 2 and 3
         ([65000, 0, 130, 1, 700], 200, 264, HALF, (128, 256)), ([65000, 0, 130, 1, 700], 64, 261, HALF, (128, 256)),
         ([65000, 0, 130, 1, 700], 72, 264, HALF, (128, 256)), ([65000, 0, 130, 1, 700], 136, 331, HALF, (128, 256))]


@pytest.mark.parametrize("sizes,cin,cout,dtype,tile", [(s, i, o, d, t) for s, i, o, ds, t in TILES for d in ds])
def test_gated_tiles(dmr, sizes, cin, cout, dtype, tile):
    say(f"[gpu] gated {dtype} {cin}->{cout} sizes {sizes} tile {tile}")
    plan = dmr.dmr_grouped_gated_linear_plan(sum(sizes), len(sizes), cin, cout, TORCH[dtype])
    assert (plan["columns"], plan["rows"]) == tile and not (plan["one_kernel"] and cin > 64)
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, cin, cout, dtype, cin)
    offd = torch.from_numpy(off).to(DEV)
    y = torch.full((x.shape[0], cout), float("nan"), dtype=x.dtype, device=DEV)
    dmr.dmr_grouped_gated_linear_fwd(x, offd, w, b, y)
    _check(y, gated_forward(x64, off, w64, b64), gated_forward_bound(x64, off, w64, b64, dtype), "y")
    for got, ref, bound, what in zip(_backward(dmr, x, offd, w, b, g), gated_backward(x64, off, w64, b64, g64),
                                     gated_backward_bound(x64, off, w64, b64, g64, dtype), ("gx", "gw", "gb")):
        _check(got, ref, bound, what)


# hidden widths of both forms; pieces of 128 rows and longer ones, of one and
# several iterations with a remainder; widths that are padded, whole and not
NARROW = [([128, 0, 127, 129, 1], 64, 64), ([128, 0, 127, 129, 1], 37, 53), ([128, 0, 127, 129, 1], 64, 128),
          ([128, 0, 127, 129, 1], 61, 127), ([100000, 3, 0, 31000], 64, 64), ([100000, 3, 0, 31000], 64, 128),
          ([70000, 3, 0, 20000], 33, 65), ([70000, 3, 0, 20000], 20, 36), ([1000, 40], 1, 128), ([1000, 40], 64, 1),
          ([1] * 300, 48, 80)]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("sizes,cin,cout", NARROW)
def test_gated_backward_in_one_kernel(dmr, sizes, cin, cout, dtype):
    say(f"[gpu] gated, one kernel {dtype} {cin}->{cout} sizes {sizes[:8]}")
    plan = dmr.dmr_grouped_gated_linear_plan(sum(sizes), len(sizes), cin, cout, TORCH[dtype])
    assert plan["one_kernel"] and plan["piece_rows"] == (128 if sum(sizes) <= 65536 // 2 else plan["piece_rows"])
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, cin, cout, dtype, cin)
    offd = torch.from_numpy(off).to(DEV)
    for got, ref, bound, what in zip(_backward(dmr, x, offd, w, b, g, "gelu_tanh"),
                                     gated_backward(x64, off, w64, b64, g64, "gelu_tanh"),
                                     gated_backward_bound(x64, off, w64, b64, g64, dtype, "gelu_tanh"), ("gx", "gw", "gb")):
        _check(got, ref, bound, what)


# few rows for each of many groups: the weights' gradient row by row (whole 16
# bytes and not, empty groups, one long group among them, one gradient alone)
@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("sizes,cin,cout", [([1] * 40, 200, 300), ([1, 0, 3, 2] * 12, 201, 307), ([0] * 30 + [90] + [1] * 10, 136, 500),
                                            ([2, 1] * 16, 3, 30000)])
def test_gated_backward_of_few_rows(dmr, sizes, cin, cout, dtype):
    say(f"[gpu] gated, few rows {dtype} {cin}->{cout} groups {len(sizes)}")
    assert sum(sizes) <= 4 * len(sizes) and len(sizes) * cin * cout >= 1 << 21
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, cin, cout, dtype, cin)
    offd = torch.from_numpy(off).to(DEV)
    ref = gated_backward(x64, off, w64, b64, g64)
    bound = gated_backward_bound(x64, off, w64, b64, g64, dtype)
    for grads in ((True, True, True), (False, True, False), (False, False, True)):
        for got, r, e, what in zip(_backward(dmr, x, offd, w, b, g, grads=grads), ref, bound, ("gx", "gw", "gb")):
            if got is not None:
                _check(got, r, e, what)


def test_gated_plans(dmr):
    plan = dmr.dmr_grouped_gated_linear_plan
    assert plan(1 << 20, 16, 64, 64, torch.bfloat16)["one_kernel"] and not plan(1 << 20, 16, 72, 64, torch.bfloat16)["one_kernel"]
    assert not plan(1 << 20, 16, 64, 129, torch.bfloat16)["one_kernel"]
    # the largest tiles have no form for arrays that are not aligned
    assert plan(1 << 20, 16, 256, 256, torch.bfloat16)["rows"] == 256
    assert plan(1 << 20, 16, 256, 256, torch.bfloat16, aligned=False)["rows"] == 128
    for bad in ((-1, 2, 8, 4, torch.float32), (10, 0, 8, 4, torch.float32), (10, 2, 0, 4, torch.float32),
                (10, 2, 8, 1 << 20, torch.float32), (10, 2, 8, 4, torch.float64)):
        with pytest.raises(dmr.DmrError):
            plan(*bad)
