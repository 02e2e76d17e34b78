"""Calls of the layer norms at the edges of what is allowed.

Tolerances: as in test_gpu_norms.py (oracle/norms.py)."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_norms import _check, _inputs
from oracle.norms import layer_norm_backward, layer_norm_backward_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


# a lane to a row, some, all of a wave's, and a workgroup to a row; the first
# group begins inside a workgroup's rows, at their end, and workgroups later
@pytest.mark.parametrize("C", [3, 60, 64, 300, 1024, 5000])
@pytest.mark.parametrize("first,sizes,last", [(3, [17, 0, 10], 20), (1, [1], 0), (256, [64, 300], 1), (900, [40, 0, 500], 3),
                                              (40, [0, 0], 9)])
def test_norm_backward_of_groups_that_begin_after_the_first_row(dmr, first, sizes, last, C):
    say(f"[gpu] layer norm backward, {C}, rows before and behind the groups {first} {sizes} {last}")
    whole = [first, *sizes, last]
    off, (x, x64), (w, w64), _, (g, g64) = _inputs(whole, C, "float32", C)
    R, N = int(off[-1]), len(sizes)
    off, w, w64 = off[1:-1], w[1:-1].contiguous(), w64[1:-1]
    offd = torch.from_numpy(off).to(DEV)
    gx = torch.full((R, C), 7.0, device=DEV)
    gw, gb = (torch.full((N, C), float("nan"), device=DEV) for _ in range(2))
    ws = torch.empty(dmr.dmr_grouped_layer_norm_workspace_size(R, N, C, x.dtype), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)
    dmr.dmr_grouped_layer_norm_bwd(x, offd, w, g, gx, gw, gb, ws)
    mine, rest = slice(int(off[0]), int(off[-1])), off - off[0]
    args = (x64[mine], rest, w64, g64[mine])
    for got, ref, bound, what in zip((gx[mine], gw, gb), layer_norm_backward(*args), layer_norm_backward_bound(*args, "float32"),
                                     ("gx", "gw", "gb")):
        _check(got, ref, bound, what)
    assert (gx[:mine.start] == 7.0).all() and (gx[mine.stop:] == 7.0).all()
