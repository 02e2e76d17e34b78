"""The gated layers on the GPU (through the C ABI) against their oracle in 64
bits: every element within the bound derived in oracle/grouped_gated.py."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from oracle.grouped_gated import ACTIVATIONS, gated_backward, gated_backward_bound, gated_forward, gated_forward_bound

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _typed(a, dtype):
    """(device tensor of the type, the values it holds in float64)"""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


def _inputs(sizes, cin, cout, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    R, N = int(off[-1]), len(sizes)
    return (off, _typed(rng.normal(size=(R, cin)), dtype), _typed(rng.normal(size=(N, 2, cout, cin)) * scale / cin ** 0.5, dtype),
            _typed(0.3 * rng.normal(size=(N, 2, cout)), dtype), _typed(rng.normal(size=(R, cout)), dtype))


def _backward(dmr, x, off, w, b, g, act="silu", grads=(True, True, True)):
    R, cin = x.shape
    N, _, cout, _ = w.shape
    out = [torch.full(s, float("nan"), dtype=x.dtype, device=DEV) if on else None
           for s, on in zip(((R, cin), (N, 2, cout, cin), (N, 2, cout)), grads)]
    ws = torch.empty(dmr.dmr_grouped_gated_linear_workspace_size(R, N, cin, cout, x.dtype), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)      # NaN: nothing is read before it is written
    dmr.dmr_grouped_gated_linear_bwd(x, off, w, b, g, *out, ws, act)
    return out


def _check(got, ref, bound, what):
    got = got.to(torch.float64).cpu().numpy()
    assert got.shape == ref.shape
    err = np.abs(got - ref)
    assert (err <= bound).all(), (what, float((err / bound).max()))   # a NaN fails too


def _check_layer(dmr, sizes, cin, cout, dtype, act="silu", seed=0, scale=1.0):
    say(f"[gpu] gated {act} {dtype} {cin}->{cout} sizes {sizes if len(sizes) < 9 else (len(sizes), sum(sizes))}")
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, cin, cout, dtype, seed, scale)
    offd = torch.from_numpy(off).to(DEV)
    for bias, bias64 in ((b, b64), (None, None)):
        y = torch.full((x.shape[0], cout), float("nan"), dtype=x.dtype, device=DEV)
        dmr.dmr_grouped_gated_linear_fwd(x, offd, w, bias, y, act)
        _check(y, gated_forward(x64, off, w64, bias64, act), gated_forward_bound(x64, off, w64, bias64, dtype, act), "y")
        for got, ref, bound, what in zip(_backward(dmr, x, offd, w, bias, g, act), gated_backward(x64, off, w64, bias64, g64, act),
                                         gated_backward_bound(x64, off, w64, bias64, g64, dtype, act), ("gx", "gw", "gb")):
            _check(got, ref, bound, what)


# widths: one; odd; multiples of 8 (wide 16-bit accesses) and of 4 only
# (wide float32 ones); just under, at and over the tiles' sides
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("cin,cout", [(1, 1), (64, 3), (3, 64), (37, 19), (24, 40), (20, 12), (64, 64), (72, 64), (64, 72),
                                      (128, 16), (16, 128), (136, 120), (127, 129), (200, 264)])
def test_gated_widths(dmr, cin, cout, dtype):
    _check_layer(dmr, [0, 130, 1, 0, 77, 300, 0], cin, cout, dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes", [[1], [0, 0, 5], [1] * 70, [3, 0, 16, 1, 17], [64] * 3, [128, 256, 127],
                                   [255, 257, 1], [0] * 100 + [40] + [0] * 200 + [9], [2] * 300])
@pytest.mark.parametrize("cin,cout", [(64, 48), (96, 160), (33, 65)])
def test_gated_group_sizes(dmr, sizes, cin, cout, dtype):
    _check_layer(dmr, sizes, cin, cout, dtype, "gelu_tanh")


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("act", ACTIVATIONS)
@pytest.mark.parametrize("cin,cout,scale", [(64, 64, 1.0), (37, 53, 8.0), (130, 70, 30.0)])
def test_gated_activations(dmr, act, cin, cout, scale, dtype):
    # arguments up to about 3, 30 and 100: both tails of every activation
    _check_layer(dmr, [90, 0, 200], cin, cout, dtype, act, seed=2, scale=scale)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes,cin,cout", [([5000, 3, 0, 700, 1500], 64, 64), ([9000], 40, 24), ([20000, 20000], 16, 3),
                                            ([3000, 1, 2500], 130, 140)])
def test_gated_long_groups(dmr, sizes, cin, cout, dtype):
    _check_layer(dmr, sizes, cin, cout, dtype, "gelu", seed=3)


def test_gated_layer_of_no_rows(dmr):
    x, off, w = torch.empty((0, 8), device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV), torch.ones((3, 2, 4, 8), device=DEV)
    assert dmr.grouped_gated_linear(x, off, w).shape == (0, 4)
    gx, gw, gb = _backward(dmr, x, off, w, None, torch.empty((0, 4), device=DEV))
    assert gx.shape == (0, 8) and (gw == 0).all() and (gb == 0).all()
    assert dmr.grouped_gated_linear(x, off[:1].contiguous(), w[:0]).shape == (0, 4)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes,cin,cout", [([90, 0, 700], 48, 80), ([90, 0, 700], 64, 64), ([1, 1, 1], 200, 136)])
def test_gated_gradients_one_at_a_time(dmr, sizes, cin, cout, dtype):
    off, (x, _), (w, _), (b, _), (g, _) = _inputs(sizes, cin, cout, dtype, 4)
    offd = torch.from_numpy(off).to(DEV)
    every = _backward(dmr, x, offd, w, b, g)
    for k in range(3):
        some = _backward(dmr, x, offd, w, b, g, grads=[i == k for i in range(3)])
        assert [s is not None for s in some] == [i == k for i in range(3)]
        assert torch.equal(some[k], every[k])


@pytest.mark.parametrize("dtype", list(TORCH))
def test_gated_unaligned_arrays(dmr, dtype):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs([40, 3, 200], 64, 32, dtype, 5)
    offd = torch.from_numpy(off).to(DEV)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    y = shifted(torch.zeros((len(x64), 32), dtype=x.dtype, device=DEV))
    dmr.dmr_grouped_gated_linear_fwd(shifted(x), offd, shifted(w), shifted(b), y)
    _check(y, gated_forward(x64, off, w64, b64), gated_forward_bound(x64, off, w64, b64, dtype), "y")
    for got, ref, bound in zip(_backward(dmr, shifted(x), offd, shifted(w), shifted(b), shifted(g)),
                               gated_backward(x64, off, w64, b64, g64), gated_backward_bound(x64, off, w64, b64, g64, dtype)):
        _check(got, ref, bound, "grad")


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("cin,cout", [(64, 64), (37, 19)])
def test_gated_non_finite_values_stay_in_their_row_and_group(dmr, cin, cout, dtype):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs([33, 20, 0, 600], cin, cout, dtype, 6)
    offd = torch.from_numpy(off).to(DEV)
    x[40, 5], x[2, 0] = float("inf"), float("nan")      # groups 1 and 0
    clean = np.ones(len(x64), bool)
    clean[[2, 40]] = False
    y = dmr.grouped_gated_linear(x, offd, w, b).double().cpu().numpy()
    ref, bound = gated_forward(x64, off, w64, b64), gated_forward_bound(x64, off, w64, b64, dtype)
    assert (np.abs(y - ref)[clean] <= bound[clean]).all() and np.isnan(y[2]).all() and not np.isfinite(y[40]).any()
    gx, gw, gb = (t.double().cpu().numpy() for t in _backward(dmr, x, offd, w, b, g))
    (rx, rw, rb), (bx, bw, bb) = gated_backward(x64, off, w64, b64, g64), gated_backward_bound(x64, off, w64, b64, g64, dtype)
    assert (np.abs(gx - rx)[clean] <= bx[clean]).all() and not np.isfinite(gx[2]).any()
    for got, r, e in ((gw, rw, bw), (gb, rb, bb)):
        assert np.isnan(got[0]).all() and (np.abs(got - r)[2:] <= e[2:]).all()


@pytest.mark.parametrize("cin,cout", [(64, 64), (37, 19), (200, 136)])
def test_gated_leaves_rows_of_no_group_as_they_are(dmr, cin, cout):
    x, g, w = torch.randn((300, cin), device=DEV), torch.randn((300, cout), device=DEV), torch.randn((2, 2, cout, cin), device=DEV)
    off = torch.tensor([0, 120, 230], device=DEV)
    y = torch.full((300, cout), 7.0, device=DEV)
    dmr.dmr_grouped_gated_linear_fwd(x, off, w, None, y)
    assert (y[230:] == 7.0).all() and torch.isfinite(y).all()
    gx = torch.full((300, cin), 7.0, device=DEV)
    ws = torch.empty(dmr.dmr_grouped_gated_linear_workspace_size(300, 2, cin, cout, x.dtype), dtype=torch.uint8, device=DEV)
    dmr.dmr_grouped_gated_linear_bwd(x, off, w, None, g, gx, None, None, ws)
    assert (gx[230:] == 7.0).all() and torch.isfinite(gx).all()


def test_gated_results_repeat_and_use_the_current_stream(dmr):
    off, (x, _), (w, _), (b, _), (g, _) = _inputs([4000, 10, 3000], 64, 64, "bfloat16", 7)
    offd = torch.from_numpy(off).to(DEV)
    first = [dmr.grouped_gated_linear(x, offd, w, b)] + _backward(dmr, x, offd, w, b, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [dmr.grouped_gated_linear(x, offd, w, b)] + _backward(dmr, x, offd, w, b, g)
    side.synchronize()
    for a, c in zip(first, again):
        assert torch.equal(a, c)


def test_gated_autograd(dmr):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs([10, 0, 25], 12, 7, "float32", 8)
    offd = torch.from_numpy(off).to(DEV)
    for act in ACTIVATIONS:
        leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
        y = dmr.grouped_gated_linear(leaves[0], offd, leaves[1], leaves[2], act)
        y.backward(g.t().contiguous().t())          # a gradient that is not contiguous
        for t, r, bound in zip(leaves, gated_backward(x64, off, w64, b64, g64, act),
                               gated_backward_bound(x64, off, w64, b64, g64, "float32", act)):
            _check(t.grad, r, bound, "grad")
    w2 = w.clone().requires_grad_(True)
    dmr.grouped_gated_linear(x, offd, w2).backward(g)
    ref = gated_backward(x64, off, w64, None, g64)[1]
    _check(w2.grad, ref, gated_backward_bound(x64, off, w64, None, g64, "float32")[1], "no bias")
    assert not dmr.grouped_gated_linear(x, offd, w, b).requires_grad
    xg = x.clone().requires_grad_(True)
    (gx,) = torch.autograd.grad(dmr.grouped_gated_linear(xg, offd, w).sum(), xg, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            dmr.grouped_gated_linear(dual, offd, w)


@pytest.mark.parametrize("act", ACTIVATIONS)
def test_gated_activations_of_very_large_arguments(dmr, act):
    # a = 1e25 and -1e25 (whose squares pass float32's range), u = 1
    x, off = torch.ones((2, 1), device=DEV), torch.tensor([0, 1, 2], device=DEV)
    w = torch.tensor([[[[1e25]], [[1.0]]], [[[-1e25]], [[1.0]]]], device=DEV)
    high, slope = (1.0, 0.0) if act == "sigmoid" else (float(w[0, 0, 0, 0]), 1.0)
    for cout in (1, 130):       # both forms of the backward pass
        wide = w.expand(2, 2, cout, 1).contiguous()
        y = dmr.grouped_gated_linear(x, off, wide, None, act)
        assert (y[0] == high).all() and (y[1] == 0).all()
        _, gw, _ = _backward(dmr, x, off, wide, None, torch.ones_like(y), act)
        assert (gw[0, 0] == slope).all() and (gw[0, 1] == high).all() and (gw[1] == 0).all()


def test_gated_refusals(dmr):
    x, w = torch.zeros((4, 8), device=DEV), torch.zeros((2, 2, 3, 8), device=DEV)
    off = torch.tensor([0, 1, 4], dtype=torch.int64, device=DEV)
    y = torch.zeros((4, 3), device=DEV)
    for bad in (dict(x=x.half()), dict(x=x.double()), dict(off=off.int()), dict(off=off[:2].contiguous()), dict(w=w[..., :7]),
                dict(w=w.cpu()), dict(w=w[:, 0].contiguous()), dict(w=w[:, :1].contiguous()), dict(x=torch.zeros((8, 4), device=DEV).t()),
                dict(y=y[:3]), dict(b=torch.zeros((2, 3), device=DEV)), dict(act="relu")):
        a = dict(x=x, off=off, w=w, b=None, y=y, act="silu")
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dmr.dmr_grouped_gated_linear_fwd(a["x"], a["off"], a["w"], a["b"], a["y"], a["act"])
    with pytest.raises(ValueError):      # the backward pass needs a workspace
        dmr.dmr_grouped_gated_linear_bwd(x, off, w, None, y, torch.empty_like(x), None, None, None)
    with pytest.raises(dmr.DmrError):
        dmr.dmr_grouped_gated_linear_bwd(x, off, w, None, y, torch.empty_like(x), None, None,
                                         torch.empty(16, dtype=torch.uint8, device=DEV))


def test_gated_past_32_bit_offsets(dmr):
    # x, or y, holds more than 2^32 bytes: rows at the end, aligned and not
    for cin, cout in ((2048, 16), (2047, 3), (16, 2048)):
        R, tail = (1 << 20) + 3000, 200
        say(f"[gpu] gated {R} rows of {cin} -> {cout}")
        x = torch.zeros((R, cin), dtype=torch.bfloat16, device=DEV)
        g = torch.zeros((R, cout), dtype=torch.bfloat16, device=DEV)
        off = np.array([0, 1 << 20, R - 70, R], np.int64)
        rng = np.random.default_rng(1)
        (xt, x64), (gt, g64) = _typed(rng.normal(size=(tail, cin)), "bfloat16"), _typed(rng.normal(size=(tail, cout)), "bfloat16")
        x[R - tail:], g[R - tail:] = xt, gt
        w, w64 = _typed(rng.normal(size=(3, 2, cout, cin)) / cin ** 0.5, "bfloat16")
        offd = torch.from_numpy(off).to(DEV)
        last = np.array([0, 0, tail - 70, tail], np.int64)     # the groups of the rows that are not zero
        y = dmr.grouped_gated_linear(x, offd, w)
        _check(y[R - tail:], gated_forward(x64, last, w64), gated_forward_bound(x64, last, w64, None, "bfloat16"), "y")
        assert (y[:R - tail] == 0).all()
        grads = _backward(dmr, x, offd, w, None, g)
        ref, bound = gated_backward(x64, last, w64, None, g64), gated_backward_bound(x64, last, w64, None, g64, "bfloat16")
        _check(grads[0][R - tail:], ref[0], bound[0], "gx")
        for k in (1, 2):
            _check(grads[k], ref[k], bound[k], "gw, gb")
        del x, y, g, grads


def test_gated_layers_in_a_graph(dmr):
    off = torch.tensor([0, 300, 300, 2000], dtype=torch.int64, device=DEV)
    x, w, g = torch.randn(2000, 64, device=DEV), torch.randn(3, 2, 32, 64, device=DEV), torch.randn(2000, 32, device=DEV)

    def work():
        return [dmr.grouped_gated_linear(x, off, w)] + _backward(dmr, x, off, w, None, g)

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
        eager = work()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
