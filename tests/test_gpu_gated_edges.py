"""Calls of the gated layers at the edges of what is allowed, through the C ABI.

Tolerances: as in test_gpu_gated.py (oracle/grouped_gated.py)."""

import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_gated import _backward, _check, _inputs
from oracle.grouped_gated import gated_backward, gated_backward_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


# one kernel of both widths, the weights' gradient row by row, and the linear layer's
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,cin,cout", [(3, 64, 64), (300, 37, 128), (40, 200, 300), (2, 130, 140)])
def test_gated_backward_without_rows_needs_no_inputs(dmr, N, cin, cout, dtype):
    say(f"[gpu] gated backward of no rows, {N} groups {cin}->{cout} {dtype}, no inputs")
    code, off = dmr.DTYPES[dtype], torch.zeros(N + 1, dtype=torch.int64, device=DEV)
    gw = torch.full((N, 2, cout, cin), float("nan"), dtype=dtype, device=DEV)
    gb = torch.full((N, 2, cout), float("nan"), dtype=dtype, device=DEV)
    gx = torch.empty(16, dtype=dtype, device=DEV)       # of no rows, but not NULL
    ws = torch.empty(dmr.dmr_grouped_gated_linear_workspace_size(0, N, cin, cout, dtype), dtype=torch.uint8, device=DEV)
    for grad_x in (None, gx.data_ptr()):
        rc = dmr.lib().dmr_grouped_gated_linear_bwd(None, 0, cin, off.data_ptr(), N, None, None, cout, 0, code, None, grad_x,
                                                    gw.data_ptr(), gb.data_ptr(), ws.data_ptr(), ws.numel(),
                                                    torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0 and (gw == 0).all() and (gb == 0).all()


# few rows on average, nearly all of them one group's: aligned and not, few and many tiles
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("before,size,after,cin,cout", [(900, 3000, 400, 72, 40), (40, 65, 30, 131, 260), (2000, 8300, 1000, 67, 33),
                                                        (20, 64, 30, 136, 320), (30, 400, 100, 136, 200)])
def test_gated_backward_of_one_long_group_among_many_short_ones(dmr, before, size, after, cin, cout, dtype):
    say(f"[gpu] gated, {size} rows of one group among {before + after}, {cin}->{cout} {dtype}")
    sizes = [0, 1, 0, 2] * (before // 4) + [size] + [1, 0] * (after // 2)
    assert sum(sizes) <= 4 * len(sizes) and len(sizes) * cin * cout >= 1 << 21
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, cin, cout, dtype, cin)
    offd = torch.from_numpy(off).to(DEV)
    ref, bound = gated_backward(x64, off, w64, b64, g64), gated_backward_bound(x64, off, w64, b64, g64, dtype)
    for grads in ((True, True, True), (False, True, False), (False, False, True), (True, False, False)):
        for got, r, e, what in zip(_backward(dmr, x, offd, w, b, g, grads=grads), ref, bound, ("gx", "gw", "gb")):
            if got is not None:
                _check(got, r, e, what)


# the forms of the backward pass that lay operands out in the workspace, or take more launches than float32's
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sizes,cin,cout", [([300, 0, 1700], 64, 32), ([300, 0, 1700], 136, 72), ([1, 0, 90, 2] + [1] * 60, 136, 300)])
def test_gated_16_bit_backward_in_a_graph(dmr, sizes, cin, cout, dtype):
    say(f"[gpu] gated backward in a graph, {cin}->{cout} {dtype}")
    R, N = sum(sizes), len(sizes)
    off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], device=DEV)
    x, w, g = (torch.randn(s, device=DEV).to(dtype) for s in ((R, cin), (N, 2, cout, cin), (R, cout)))

    def work():
        return _backward(dmr, x, off, w, None, g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(4):
        x.copy_(torch.randn_like(x))
        w.copy_(torch.randn_like(w))
        eager = work()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
