"""Second derivatives of the per-group layer on the GPU, against the formula in
64 bits: with grad_x_r = W_n^T g_r, grad_W_n = sum_r g_r x_r^T and grad_b_n =
sum_r g_r, and upstream gradients hx, hw, hb of the three,

    d/dx_r = hw_n^T g_r,  d/dW_n = sum_r g_r hx_r^T,  d/dg_r = W_n hx_r + hw_n x_r + hb_n,

each a product of the layer, within that product's bound
(oracle/grouped_linear.py); the last is a sum of two rounded ones."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from oracle.grouped_linear import (UNIT, backward_error_bound, forward_error_bound, grouped_linear_backward,
                                   grouped_linear_forward)

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _check(got, ref, bound, what):
    err = np.abs(got.detach().to(torch.float64).cpu().numpy() - ref)
    assert (err <= bound).all(), (what, float((err / bound).max()))   # a NaN fails too


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes,cin,cout", [([10, 0, 25], 12, 7), ([200, 1, 0, 700], 64, 48), ([1] * 9, 33, 65)])
def test_second_derivatives(dmr, sizes, cin, cout, dtype):
    say(f"[gpu] second derivatives {dtype} {cin}->{cout} sizes {sizes}")
    rng = np.random.default_rng(cin)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    R, N = int(off[-1]), len(sizes)
    shapes = dict(x=(R, cin), w=(N, cout, cin), b=(N, cout), g=(R, cout), hx=(R, cin), hw=(N, cout, cin), hb=(N, cout))
    t = {k: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(TORCH[dtype]) for k, s in shapes.items()}
    v = {k: a.to(torch.float64).numpy() for k, a in t.items()}
    t = {k: a.to(DEV).requires_grad_(k in "xwbg") for k, a in t.items()}
    offd = torch.from_numpy(off).to(DEV)
    grads = torch.autograd.grad(dmr.grouped_linear(t["x"], offd, t["w"], t["b"]), (t["x"], t["w"], t["b"]), t["g"],
                                create_graph=True)
    dx, dw, dg = torch.autograd.grad(grads, (t["x"], t["w"], t["g"]), (t["hx"], t["hw"], t["hb"]), retain_graph=True)
    _check(dx, grouped_linear_backward(v["x"], off, v["hw"], v["g"])[0],
           backward_error_bound(v["x"], off, v["hw"], v["g"], dtype)[0], "dx")
    _check(dw, grouped_linear_backward(v["hx"], off, v["w"], v["g"])[1],
           backward_error_bound(v["hx"], off, v["w"], v["g"], dtype)[1], "dw")
    ref = grouped_linear_forward(v["hx"], off, v["w"], v["hb"]) + grouped_linear_forward(v["x"], off, v["hw"])
    bound = (forward_error_bound(v["hx"], off, v["w"], v["hb"], dtype) + forward_error_bound(v["x"], off, v["hw"], None, dtype))
    _check(dg, ref, bound + UNIT[dtype] * (np.abs(ref) + bound), "dg")
    # of the bias's gradient alone: every row gets its group's, exactly
    only = torch.autograd.grad(grads[2], t["g"], t["hb"], retain_graph=True)[0]
    assert torch.equal(only, t["hb"].repeat_interleave(torch.tensor(sizes, device=DEV), dim=0))


def test_a_loss_with_a_penalty_on_its_gradients(dmr):
    # against the same loss written with torch, in float64 on the CPU
    rng = np.random.default_rng(5)
    sizes, cin, cout = [30, 0, 12], 8, 5
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int64)
    leaves = [torch.from_numpy(rng.normal(size=s)) for s in ((42, cin), (3, cout, cin), (3, cout))]
    group = torch.repeat_interleave(torch.arange(3), torch.tensor(sizes))

    def gradients(layer, x, w, b):
        y = torch.tanh(layer(x, w, b))
        first = torch.autograd.grad((y ** 2).mean(), (x, w, b), create_graph=True)
        return torch.autograd.grad((y ** 2).mean() + sum((f ** 2).sum() for f in first), (x, w, b))

    want = gradients(lambda x, w, b: torch.bmm(w[group], x[:, :, None])[:, :, 0] + b[group],
                     *[t.clone().requires_grad_(True) for t in leaves])
    got = gradients(lambda x, w, b: dmr.grouped_linear(x, off.to(DEV), w, b),
                    *[t.float().to(DEV).requires_grad_(True) for t in leaves])
    for a, c in zip(got, want):
        # some hundred roundings of 2^-24 along the way
        assert torch.linalg.vector_norm(a.cpu().double() - c) < 2.0 ** -16 * torch.linalg.vector_norm(c)
