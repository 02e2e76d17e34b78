"""How the gated layers' backward pass cuts the rows (host functions only, so
these run without a GPU)."""

import os

import pytest
import torch

HALF, ALL = (torch.float16, torch.bfloat16), (torch.float16, torch.bfloat16, torch.float32)


@pytest.fixture(scope="module")
def dmr():
    import differentiable_mesh_rasterization_amd as pkg

    if not os.path.exists(pkg.LIB_PATH):
        from differentiable_mesh_rasterization_amd import build

        build.build()
    return pkg


# the batches of test_gpu_gated_tiles.py: short ones in pieces of 128 rows, long
# ones in longer pieces, of several iterations of 64 or 128 rows
@pytest.mark.parametrize("sizes,cin,cout,types,rows", [
    ([128, 0, 127, 129, 1], 64, 64, ALL, 128), ([128, 0, 127, 129, 1], 61, 127, ALL, 128), ([1] * 300, 48, 80, ALL, 128),
    ([100000, 3, 0, 31000], 64, 64, HALF, 512), ([100000, 3, 0, 31000], 64, 64, (torch.float32,), 256),
    ([100000, 3, 0, 31000], 64, 128, ALL, 512), ([70000, 3, 0, 20000], 33, 65, ALL, 384),
    ([70000, 3, 0, 20000], 20, 36, HALF, 384), ([70000, 3, 0, 20000], 20, 36, (torch.float32,), 256),
])
def test_pieces_of_narrow_layers(dmr, sizes, cin, cout, types, rows):
    for dtype in types:
        plan = dmr.dmr_grouped_gated_linear_plan(sum(sizes), len(sizes), cin, cout, dtype)
        assert plan["one_kernel"] and plan["piece_rows"] == rows
