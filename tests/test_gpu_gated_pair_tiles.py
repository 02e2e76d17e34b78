"""Every tile that the products with [da du] as pairs take in 16-bit layers, each
asserted to be the one that the call takes (dmr_grouped_linear_plan of twice the
outputs): the rows' gradient alone, the weights' alone, and both.

Tolerances: as in test_gpu_gated.py (oracle/grouped_gated.py)."""

import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_gated import _backward, _check, _inputs
from oracle.grouped_gated import gated_backward, gated_backward_bound

pytestmark = pytest.mark.gpu

ROWS, WEIGHTS, BOTH = (True, False, False), (False, True, True), (True, True, True)


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


# (sizes, cin, cout, gradients, tile of grad_x: columns and rows, side of the
# weight's); steps of 64 values of k that end inside, rows that end inside a
# tile, and widths of no whole 16 bytes
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("sizes,cin,cout,grads,rows,side", [
    ([5, 0, 16, 1], 200, 140, ROWS, (64, 16), None), ([5, 0, 16, 1], 203, 139, BOTH, (64, 16), None),
    ([3000, 0, 77], 16, 130, ROWS, (16, 128), None), ([3000, 0, 77], 13, 131, ROWS, (16, 128), None),
    ([3000, 0, 77], 64, 130, ROWS, (64, 128), None), ([3000, 0, 77], 63, 131, ROWS, (64, 128), None),
    ([65800, 0, 77], 64, 130, ROWS, (64, 256), None), ([65800, 0, 77], 61, 131, ROWS, (64, 256), None),
    ([17000, 0, 77], 200, 140, ROWS, (128, 128), None), ([17000, 0, 77], 203, 139, ROWS, (128, 128), None),
    ([3000, 0, 77], 200, 140, BOTH, (64, 128), None), ([3000, 0, 77], 15, 139, BOTH, (16, 128), None),
    ([3000, 0, 77], 200, 140, WEIGHTS, None, 128), ([3000, 0, 77], 203, 139, WEIGHTS, None, 128),
    ([1500, 700, 0, 900, 1100, 800, 1300, 800], 1024, 264, BOTH, (256, 256), 256),
])
def test_products_with_pairs(dmr, sizes, cin, cout, grads, rows, side, dtype):
    say(f"[gpu] gated, pairs {dtype} {cin}->{cout} sizes {sizes} tiles {rows} {side}")
    aligned = cin % 8 == 0 and cout % 8 == 0
    plan = dmr.dmr_grouped_linear_plan(sum(sizes), len(sizes), cin, 2 * cout, getattr(torch, dtype), aligned)
    assert rows is None or (plan["grad_x_columns"], plan["grad_x_rows"]) == rows
    assert side is None or plan["grad_weight_side"] == side
    assert grads != BOTH or plan["together"] == (side is None)
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, cin, cout, dtype, cin)
    ref, bound = gated_backward(x64, off, w64, b64, g64), gated_backward_bound(x64, off, w64, b64, g64, dtype)
    for got, r, e, what in zip(_backward(dmr, x, torch.from_numpy(off).to(DEV), w, b, g, grads=grads), ref, bound, ("gx", "gw", "gb")):
        if got is not None:
            _check(got, r, e, what)
