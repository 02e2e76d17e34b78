"""The per-group linear layers and the orthogonalised updates on the GPU
(through the C ABI) against their oracles in 64 bits.

Every element of the layer and its gradients must lie within the binary32
bound of a sum of that many products, plus one rounding to the output's type
(oracle/grouped_linear.py: sum_error_bound). The orthogonalised updates must
lie within twice the Frobenius error that rounded factors lead to expect
(oracle/orthogonalize.py: expected_error, which is 1/2 to 12 times what such
an iteration shows): factors rounded to 23 bits for float32 and float16
results, to 12 for bfloat16 ones."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from oracle.grouped_linear import (backward_error_bound, forward_error_bound, grouped_linear_backward,
                                   grouped_linear_forward)
from oracle.orthogonalize import expected_error, orthogonalize

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _typed(a, dtype):
    """(device tensor of the type, the values it holds in float64)"""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


def _off(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)


def _layer_inputs(sizes, cin, cout, dtype, seed):
    rng = np.random.default_rng(seed)
    off = _off(sizes)
    R, N = int(off[-1]), len(sizes)
    return (off, _typed(rng.normal(size=(R, cin)), dtype), _typed(rng.normal(size=(N, cout, cin)), dtype),
            _typed(rng.normal(size=(N, cout)), dtype), _typed(rng.normal(size=(R, cout)), dtype))


def _backward(dmr, x, off, w, g, grads=(True, True, True)):
    R, cin = x.shape
    N, cout, _ = w.shape
    out = [torch.full(s, float("nan"), dtype=x.dtype, device=DEV) if on else None
           for s, on in zip(((R, cin), (N, cout, cin), (N, cout)), grads)]
    ws = torch.empty(dmr.dmr_grouped_linear_workspace_size(R, N, cin, cout, x.dtype), dtype=torch.uint8, device=DEV)
    dmr.dmr_grouped_linear_bwd(x, off, w, g, *out, ws)
    return out


def _check(got, ref, bound, what):
    got = got.to(torch.float64).cpu().numpy()
    assert got.shape == ref.shape
    err = np.abs(got - ref)
    assert (err <= bound).all(), (what, float((err / bound).max()))   # a NaN fails too


def _check_layer(dmr, sizes, cin, cout, dtype, seed=0):
    say(f"[gpu] grouped_linear {dtype} {cin}->{cout} sizes {sizes if len(sizes) < 9 else (len(sizes), sum(sizes))}")
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _layer_inputs(sizes, cin, cout, dtype, seed)
    offd = torch.from_numpy(off).to(DEV)
    for bias, bias64 in ((b, b64), (None, None)):
        y = torch.full((x.shape[0], cout), float("nan"), dtype=x.dtype, device=DEV)
        dmr.dmr_grouped_linear_fwd(x, offd, w, bias, y)
        _check(y, grouped_linear_forward(x64, off, w64, bias64), forward_error_bound(x64, off, w64, bias64, dtype), "y")
    for got, ref, bound, what in zip(_backward(dmr, x, offd, w, g), grouped_linear_backward(x64, off, w64, g64),
                                     backward_error_bound(x64, off, w64, g64, dtype), ("gx", "gw", "gb")):
        _check(got, ref, bound, what)


# widths: one; a vertex offset; odd; a multiple of 8 (wide 16-bit loads) and
# of 4 only (wide float32 loads); just under, at and over the tile sides
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("cin,cout", [(1, 1), (64, 3), (3, 64), (37, 19), (24, 40), (20, 12), (64, 64), (72, 64),
                                      (128, 16), (16, 128), (136, 120), (127, 129), (200, 264)])
def test_layer_widths(dmr, cin, cout, dtype):
    _check_layer(dmr, [0, 130, 1, 0, 77, 300, 0], cin, cout, dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes", [[1], [0, 0, 5], [1] * 70, [3, 0, 16, 1, 17], [64] * 3, [128, 256, 127],
                                   [255, 257, 1], [0] * 100 + [40] + [0] * 200 + [9], [2] * 300])
@pytest.mark.parametrize("cin,cout", [(64, 48), (96, 160), (33, 65)])
def test_layer_group_sizes(dmr, sizes, cin, cout, dtype):
    _check_layer(dmr, sizes, cin, cout, dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes,cin,cout", [([5000, 3, 0, 700, 1500], 64, 64), ([9000], 40, 24), ([20000, 20000], 16, 3),
                                            ([3000, 1, 2500], 130, 140)])
def test_layer_long_groups_are_cut_and_joined(dmr, sizes, cin, cout, dtype):
    _check_layer(dmr, sizes, cin, cout, dtype, seed=3)


def test_layer_of_no_rows(dmr):
    x = torch.empty((0, 8), device=DEV)
    w = torch.ones((3, 4, 8), device=DEV)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    assert dmr.grouped_linear(x, off, w).shape == (0, 4)
    gx, gw, gb = _backward(dmr, x, off, w, torch.empty((0, 4), device=DEV))
    assert gx.shape == (0, 8) and (gw == 0).all() and (gb == 0).all()
    # no group at all
    none = dmr.grouped_linear(x, off[:1].contiguous(), w[:0])
    assert none.shape == (0, 4)


@pytest.mark.parametrize("dtype", list(TORCH))
def test_layer_gradients_one_at_a_time(dmr, dtype):
    off, (x, _), (w, _), _, (g, _) = _layer_inputs([90, 0, 700], 48, 80, dtype, 4)
    offd = torch.from_numpy(off).to(DEV)
    every = _backward(dmr, x, offd, w, g)
    for k in range(3):
        some = _backward(dmr, x, offd, w, g, [i == k for i in range(3)])
        assert [s is not None for s in some] == [i == k for i in range(3)]
        assert torch.equal(some[k], every[k])


# the gradients of the rows and of the weights each in a launch of its own:
# rows of few per group, narrow, wide and unaligned; weights of one small tile
# and of larger ones; and, of more tiles than one launch of both takes, together
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes,cin,cout", [([3, 0, 16, 1, 17], 64, 48), ([3, 0, 16, 1, 17], 37, 65), ([200, 0, 333], 16, 72),
                                            ([200, 0, 333], 13, 19), ([200, 0, 333], 64, 24), ([200, 0, 333], 61, 130),
                                            ([200, 0, 333], 136, 200), ([5, 300], 1000, 1100), ([1] * 12, 777, 808)])
@pytest.mark.parametrize("grads", [(True, False, False), (False, True, True), (True, True, True)])
def test_layer_gradients_apart(dmr, sizes, cin, cout, dtype, grads):
    off, (x, x64), (w, w64), _, (g, g64) = _layer_inputs(sizes, cin, cout, dtype, 6)
    got = _backward(dmr, x, torch.from_numpy(off).to(DEV), w, g, grads)
    for v, ref, bound, what in zip(got, grouped_linear_backward(x64, off, w64, g64),
                                   backward_error_bound(x64, off, w64, g64, dtype), ("gx", "gw", "gb")):
        if v is not None:
            _check(v, ref, bound, what)


@pytest.mark.parametrize("dtype", list(TORCH))
def test_layer_unaligned_arrays(dmr, dtype):
    # arrays that start one element past a 16-byte boundary, of widths that
    # would allow wide loads
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _layer_inputs([40, 3], 64, 32, dtype, 5)
    offd = torch.from_numpy(off).to(DEV)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    y = shifted(torch.zeros((43, 32), dtype=x.dtype, device=DEV))
    dmr.dmr_grouped_linear_fwd(shifted(x), offd, shifted(w), shifted(b), y)
    _check(y, grouped_linear_forward(x64, off, w64, b64), forward_error_bound(x64, off, w64, b64, dtype), "y")
    for got, ref, bound in zip(_backward(dmr, shifted(x), offd, shifted(w), shifted(g)),
                               grouped_linear_backward(x64, off, w64, g64), backward_error_bound(x64, off, w64, g64, dtype)):
        _check(got, ref, bound, "grad")


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("cin,cout", [(64, 64), (37, 19)])
def test_layer_non_finite_values_stay_in_their_row_and_group(dmr, cin, cout, dtype):
    sizes = [33, 20, 0, 600]
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _layer_inputs(sizes, cin, cout, dtype, 6)
    offd = torch.from_numpy(off).to(DEV)
    x[40, 5] = float("inf")       # group 1
    x[2, 0] = float("nan")        # group 0
    y = dmr.grouped_linear(x, offd, w, b).double().cpu().numpy()
    clean = np.ones(len(y), bool)
    clean[[2, 40]] = False
    ref = grouped_linear_forward(x64, off, w64, b64)
    bound = forward_error_bound(x64, off, w64, b64, dtype)
    assert (np.abs(y - ref)[clean] <= bound[clean]).all()
    assert np.isnan(y[2]).all()
    assert (y[40] == np.where(w64[1][:, 5] > 0, np.inf, -np.inf)).all()
    gx, gw, gb = (t.double().cpu().numpy() for t in _backward(dmr, x, offd, w, g))
    rx, rw, rb = grouped_linear_backward(x64, off, w64, g64)
    bx, bw, bb = backward_error_bound(x64, off, w64, g64, dtype)
    assert (np.abs(gx - rx) <= bx).all() and (np.abs(gb - rb) <= bb).all()
    assert np.isnan(gw[0][:, 0]).all() and not np.isfinite(gw[1][:, 5]).any()
    fine = np.ones(gw.shape, bool)
    fine[0, :, 0] = fine[1, :, 5] = False
    assert (np.abs(gw - rw)[fine] <= bw[fine]).all()


def test_layer_results_repeat_and_use_the_current_stream(dmr):
    off, (x, _), (w, _), (b, _), (g, _) = _layer_inputs([4000, 10, 3000], 64, 64, "float32", 7)
    offd = torch.from_numpy(off).to(DEV)
    first = [dmr.grouped_linear(x, offd, w, b)] + _backward(dmr, x, offd, w, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [dmr.grouped_linear(x, offd, w, b)] + _backward(dmr, x, offd, w, g)
    side.synchronize()
    for a, c in zip(first, again):
        assert torch.equal(a, c)


def test_layer_autograd(dmr):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _layer_inputs([10, 0, 25], 12, 7, "float32", 8)
    offd = torch.from_numpy(off).to(DEV)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = dmr.grouped_linear(leaves[0], offd, leaves[1], leaves[2])
    y.backward(g.t().contiguous().t())          # a gradient that is not contiguous
    ref = grouped_linear_backward(x64, off, w64, g64)
    for t, r, bound in zip(leaves, ref, backward_error_bound(x64, off, w64, g64, "float32")):
        _check(t.grad, r, bound, "grad")
    # only some arguments need one; and none does
    w2 = w.clone().requires_grad_(True)
    dmr.grouped_linear(x, offd, w2).backward(g)
    assert torch.equal(w2.grad, leaves[1].grad)
    assert not dmr.grouped_linear(x, offd, w, b).requires_grad


def test_layer_refusals(dmr):
    x, w = torch.zeros((4, 8), device=DEV), torch.zeros((2, 3, 8), device=DEV)
    off = torch.tensor([0, 1, 4], dtype=torch.int64, device=DEV)
    y = torch.zeros((4, 3), device=DEV)
    for bad in (dict(x=x.half()), dict(x=x.double()), dict(off=off.int()), dict(off=off[:2].contiguous()), dict(w=w[:, :, :7]),
                dict(w=w.cpu()), dict(x=torch.zeros((8, 4), device=DEV).t()), dict(y=y[:3]), dict(b=torch.zeros(3, device=DEV))):
        a = dict(x=x, off=off, w=w, b=None, y=y)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dmr.dmr_grouped_linear_fwd(a["x"], a["off"], a["w"], a["b"], a["y"])
    with pytest.raises(TypeError):
        dmr.grouped_linear(x.double(), off, w.double())
    with pytest.raises(ValueError):      # the gradient of the weight needs a workspace
        dmr.dmr_grouped_linear_bwd(x, off, w, y, None, torch.empty_like(w), None, None)
    with pytest.raises(dmr.DmrError):
        dmr.dmr_grouped_linear_bwd(x, off, w, y, None, torch.empty_like(w), None,
                                   torch.empty(16, dtype=torch.uint8, device=DEV))


# ----------------------------------------------------------------------------

FACTOR = {"float32": (2.0 ** -23, 2.0 ** -24), "float16": (2.0 ** -23, 2.0 ** -11), "bfloat16": (2.0 ** -12, 2.0 ** -8)}


def _check_update(got, u64, dtype, steps=5, eps=1e-7):
    got = got.to(torch.float64).cpu().numpy()
    for k in range(len(u64)):
        ref = orthogonalize(u64[k], steps, eps)
        err, expect = np.linalg.norm(got[k] - ref), expected_error(u64[k], steps, eps, *FACTOR[dtype])
        assert err <= 2 * expect, (k, err / expect)    # a NaN fails too


# one entry, rows, columns; tiles of 16 and their neighbours; the largest
# matrices that one workgroup holds and the first that it does not; padded
# and whole 64s and 128s, wide and tall
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("m,n", [(1, 1), (1, 5), (7, 1), (3, 64), (64, 3), (16, 16), (17, 33), (64, 64), (64, 65), (65, 64),
                                 (64, 400), (65, 65), (100, 300), (300, 100), (130, 70), (256, 256), (192, 640),
                                 (321, 129), (16, 3000)])
def test_update_sizes(dmr, m, n, dtype):
    say(f"[gpu] orthogonalize {dtype} {m}x{n}")
    u, u64 = _typed(np.random.default_rng(m * 1000 + n).normal(size=(2, m, n)) * 1e-3, dtype)
    _check_update(dmr.orthogonalize(u), u64, dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
def test_update_of_many_matrices_takes_the_large_tiles(dmr, dtype):
    u, u64 = _typed(np.random.default_rng(5).normal(size=(24, 150, 400)), dtype)
    got = dmr.orthogonalize(u)
    _check_update(got[::5], u64[::5], dtype)
    assert torch.equal(got, dmr.orthogonalize(u))
    one = torch.cat([dmr.orthogonalize(u[k:k + 1]) for k in (0, 23)])
    _check_update(one, u64[[0, 23]], dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("m,n", [(20, 30), (150, 90)])
@pytest.mark.parametrize("steps", [1, 2, 8])
def test_update_steps(dmr, m, n, steps, dtype):
    u, u64 = _typed(np.random.default_rng(steps).normal(size=(3, m, n)), dtype)
    _check_update(dmr.orthogonalize(u, steps), u64, dtype, steps)


@pytest.mark.parametrize("m,n", [(20, 30), (150, 90)])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e-7, 1e18, 1e36])
def test_update_of_very_small_and_large_values(dmr, m, n, scale):
    # far below eps the result is linear in the update; squares of large
    # values pass float32's range, their root does not
    u, u64 = _typed(np.random.default_rng(9).normal(size=(1, m, n)) * scale, "float32")
    _check_update(dmr.orthogonalize(u), u64, "float32")


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("m,n", [(8, 12), (100, 260)])
def test_update_of_zeros_and_of_non_finite_values(dmr, m, n, dtype):
    u, u64 = _typed(np.random.default_rng(10).normal(size=(4, m, n)), dtype)
    u[0] = 0
    u[2, 1, 3] = float("inf")
    u[3, m - 1, n - 1] = float("nan")
    got = dmr.orthogonalize(u)
    assert (got[0] == 0).all() and torch.isnan(got[2:]).all()
    _check_update(got[1:2], u64[1:2], dtype)


def test_update_of_a_matrix_of_low_rank(dmr):
    rng = np.random.default_rng(11)
    for m, n in ((48, 60), (140, 200)):
        u, u64 = _typed(rng.normal(size=(1, m, 2)) @ rng.normal(size=(1, 2, n)), "float32")
        _check_update(dmr.orthogonalize(u), u64, "float32")


def test_update_shapes_streams_and_refusals(dmr):
    u = torch.randn(33, 21, device=DEV)
    assert torch.equal(dmr.orthogonalize(u), dmr.orthogonalize(u[None])[0])
    assert dmr.orthogonalize(torch.empty((0, 5, 6), device=DEV)).shape == (0, 5, 6)
    big = torch.randn(2, 200, 300, device=DEV)
    first = dmr.orthogonalize(big)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = dmr.orthogonalize(big)
    side.synchronize()
    assert torch.equal(first, again)
    ws = torch.empty(dmr.dmr_orthogonalize_workspace_size(2, 200, 300, torch.float32), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(big)
    for bad in (dict(update=big.double()), dict(update=big.transpose(1, 2)), dict(out=out[:1]), dict(out=out.half()),
                dict(update=big[0])):
        a = dict(update=big, out=out)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dmr.dmr_orthogonalize(a["update"], a["out"], ws)
    for kw in (dict(steps=0), dict(steps=65), dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(dmr.DmrError):
            dmr.dmr_orthogonalize(big, out, ws, **kw)
    with pytest.raises(dmr.DmrError):
        dmr.dmr_orthogonalize(big, out, ws[:256])


def test_layer_of_very_many_groups(dmr):
    # more groups than a launch has places in one grid dimension
    sizes = (np.arange(70000) % 3 == 0).astype(np.int64) * 2
    _check_layer(dmr, list(sizes), 8, 8, "float32")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_layer_past_32_bit_offsets(dmr, dtype):
    # x holds more than 2^32 bytes: rows at the end, aligned and not
    for cin, cout in ((2048, 16), (2047, 3)):
        R = (1 << 20) + 3000
        say(f"[gpu] grouped_linear {dtype} {R} rows of {cin}")
        x = torch.zeros((R, cin), dtype=TORCH[dtype], device=DEV)
        off = np.array([0, 1 << 20, R - 70, R], np.int64)
        tail = 200
        xt, x64 = _typed(np.random.default_rng(1).normal(size=(tail, cin)), dtype)
        x[R - tail:] = xt
        w, w64 = _typed(np.random.default_rng(2).normal(size=(3, cout, cin)), dtype)
        g = torch.zeros((R, cout), dtype=TORCH[dtype], device=DEV)
        gt, g64 = _typed(np.random.default_rng(3).normal(size=(tail, cout)), dtype)
        g[R - tail:] = gt
        offd = torch.from_numpy(off).to(DEV)
        last = np.array([0, 0, tail - 70, tail], np.int64)     # the groups of the rows that are not zero
        y = dmr.grouped_linear(x, offd, w)
        _check(y[R - tail:], grouped_linear_forward(x64, last, w64), forward_error_bound(x64, last, w64, None, dtype), "y")
        assert (y[:R - tail] == 0).all()
        grads = _backward(dmr, x, offd, w, g)
        ref, bound = grouped_linear_backward(x64, last, w64, g64), backward_error_bound(x64, last, w64, g64, dtype)
        _check(grads[0][R - tail:], ref[0], bound[0], "gx")
        for k in (1, 2):
            _check(grads[k], ref[k], bound[k], "gw, gb")
        del x, y, g, grads


def test_layers_and_updates_in_a_graph(dmr):
    off = torch.tensor([0, 300, 300, 2000], dtype=torch.int64, device=DEV)
    x, w, g = torch.randn(2000, 64, device=DEV), torch.randn(3, 32, 64, device=DEV), torch.randn(2000, 32, device=DEV)
    u = torch.randn(2, 100, 200, device=DEV)

    def work():
        y = dmr.grouped_linear(x, off, w)
        return [y, dmr.orthogonalize(u), dmr.orthogonalize(w)] + _backward(dmr, x, off, w, g)

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
        u.copy_(torch.randn_like(u))
        eager = work()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
