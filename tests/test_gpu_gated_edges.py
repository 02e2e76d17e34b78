"""Calls of the gated layers at the edges of what is allowed, through the C ABI."""

import pytest
import torch

from gpu_util import DEV, require_gpu, say

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
