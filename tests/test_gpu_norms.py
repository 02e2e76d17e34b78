"""Layer norms with one scale and shift per group, and norms and clipping of
gradients over many tensors, on the GPU (through the C ABI) against their
oracle in 64 bits.

Every element of y and of the gradients must lie within the binary32 bound
derived in oracle/norms.py plus one rounding to the output's type; clipped
values within the roundings of factor, product and type."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from oracle.norms import (clip_bound, clip_grad_norm, layer_norm_backward, layer_norm_backward_bound, layer_norm_forward,
                          layer_norm_forward_bound)

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _typed(a, dtype):
    """(device tensor of the type, the values it holds in float64)"""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


def _inputs(sizes, C, dtype, seed, mean=0.5):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    R, N = int(off[-1]), len(sizes)
    x = rng.normal(size=(R, C)) * np.exp(rng.normal(size=(R, 1))) + mean * rng.normal(size=(R, 1))
    return (off, _typed(x, dtype), _typed(1 + 0.3 * rng.normal(size=(N, C)), dtype), _typed(rng.normal(size=(N, C)), dtype),
            _typed(rng.normal(size=(R, C)), dtype))


def _backward(dmr, x, off, w, g, grads=(True, True, True), eps=1e-5):
    R, C = x.shape
    N = len(off) - 1
    out = [torch.full(s, float("nan"), dtype=x.dtype, device=DEV) if on else None
           for s, on in zip(((R, C), (N, C), (N, C)), grads)]
    ws = torch.empty(dmr.dmr_grouped_layer_norm_workspace_size(R, N, C, x.dtype), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)      # NaN: nothing is read before it is written
    dmr.dmr_grouped_layer_norm_bwd(x, off, w, g, *out, ws, eps)
    return out


def _check(got, ref, bound, what):
    got = got.to(torch.float64).cpu().numpy()
    assert got.shape == ref.shape
    err = np.abs(got - ref)
    assert (err <= bound).all(), (what, float((err / bound).max()))   # a NaN fails too


def _check_norm(dmr, sizes, C, dtype, seed=0, mean=0.5, eps=1e-5):
    say(f"[gpu] layer norm {dtype} {C} sizes {sizes if len(sizes) < 9 else (len(sizes), sum(sizes))}")
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs(sizes, C, dtype, seed, mean)
    offd = torch.from_numpy(off).to(DEV)
    for weight, weight64, bias, bias64 in ((w, w64, b, b64), (None, None, b, b64), (w, w64, None, None), (None,) * 4):
        y = torch.full(x.shape, float("nan"), dtype=x.dtype, device=DEV)
        dmr.dmr_grouped_layer_norm_fwd(x, offd, weight, bias, y, eps)
        _check(y, layer_norm_forward(x64, off, weight64, bias64, eps),
               layer_norm_forward_bound(x64, off, weight64, bias64, dtype, eps), "y")
    for weight, weight64 in ((w, w64), (None, None)):
        for got, ref, bound, what in zip(_backward(dmr, x, offd, weight, g, eps=eps),
                                         layer_norm_backward(x64, off, weight64, g64, eps),
                                         layer_norm_backward_bound(x64, off, weight64, g64, dtype, eps), ("gx", "gw", "gb")):
            _check(got, ref, bound, what)


# widths: one lane and 2, 4 .. 64 lanes a row, 2, 4 and 8 parts a lane, and a
# workgroup a row; whole 16 bytes, odd, and just under and over each
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("C", [1, 2, 3, 4, 7, 8, 9, 16, 19, 24, 32, 37, 64, 65, 120, 128, 130, 200, 256, 257, 500, 512, 513,
                               1000, 1024, 1027, 2048, 2049, 4096, 4100, 9001])
def test_norm_widths(dmr, C, dtype):
    _check_norm(dmr, [0, 130, 1, 0, 77, 0] if C <= 512 else [0, 30, 1, 0, 9, 0], C, dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes", [[1], [0, 0, 5], [1] * 70, [3, 0, 16, 1, 17], [64] * 3, [128, 256, 127], [0] * 100 + [40] + [0] * 200 + [9],
                                   [2] * 300, [5000, 3, 0, 700, 1500], [9000], [1, 8000, 1], [4096, 0, 4096]])
@pytest.mark.parametrize("C", [3, 64, 100, 300])
def test_norm_group_sizes(dmr, sizes, C, dtype):
    _check_norm(dmr, sizes, C, dtype, seed=1)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("sizes,C", [([70000, 3, 0, 66000], 8), ([200000, 1, 17632], 64), ([3000, 0, 9000, 2], 1024),
                                     ([2500, 1, 0, 600], 4200), ([300, 5], 9001)])
def test_norm_sums_over_many_workgroups(dmr, sizes, C, dtype):
    _check_norm(dmr, sizes, C, dtype, seed=2)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("C", [37, 64, 1024, 5000])
@pytest.mark.parametrize("mean,eps", [(30.0, 1e-5), (1000.0, 1e-3), (0.0, 1e-12), (0.0, 10.0)])
def test_norm_of_rows_far_from_zero_and_of_other_eps(dmr, C, mean, eps, dtype):
    _check_norm(dmr, [20, 0, 33], C, dtype, seed=3, mean=mean, eps=eps)


def test_norm_keeps_the_digits_of_rows_far_from_zero(dmr):
    # a mean 2^18 times the deviations: the rounded mean alone would be off by
    # 2^-7 of them, the corrected one is not (the deviations are exact here);
    # the reference takes the values as float32 holds them
    x64 = 2.0 ** 14 + np.random.default_rng(4).integers(-64, 65, size=(50, 64)) * 2.0 ** -10
    x, x64 = _typed(x64, "float32")
    off = torch.tensor([0, 50], device=DEV)
    for C in (64, 63):
        y = dmr.grouped_layer_norm(x[:, :C].contiguous(), off, eps=1e-12).double().cpu().numpy()
        ref = layer_norm_forward(x64[:, :C], [0, 50], eps=1e-12)
        # numerator, root and factors: 16 roundings of the largest |h| at most
        assert np.abs(y - ref).max() <= 16 * 2.0 ** -23 * np.abs(ref).max()


@pytest.mark.parametrize("dtype", list(TORCH))
def test_norm_of_equal_values_and_of_zeros(dmr, dtype):
    x, x64 = _typed(np.array([[5.0] * 40, [0.0] * 40, [-3.0] * 40]), dtype)
    b, b64 = _typed(np.linspace(-1, 1, 40)[None], dtype)
    off = torch.tensor([0, 3], device=DEV)
    y = dmr.grouped_layer_norm(x, off, torch.ones_like(b), b)
    assert (y == b).all()


@pytest.mark.parametrize("dtype", list(TORCH))
def test_norm_gradients_one_at_a_time(dmr, dtype):
    for sizes, C in (([90, 0, 700], 48), ([30, 0, 70], 4500)):
        off, (x, _), (w, _), _, (g, _) = _inputs(sizes, C, dtype, 4)
        offd = torch.from_numpy(off).to(DEV)
        every = _backward(dmr, x, offd, w, g)
        for k in range(3):
            some = _backward(dmr, x, offd, w, g, [i == k for i in range(3)])
            assert [s is not None for s in some] == [i == k for i in range(3)]
            assert torch.equal(some[k], every[k])


def test_norm_of_no_rows(dmr):
    x, off = torch.empty((0, 8), device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    assert dmr.grouped_layer_norm(x, off).shape == (0, 8)
    gx, gw, gb = _backward(dmr, x, off, None, x)
    assert gx.shape == (0, 8) and (gw == 0).all() and (gb == 0).all()
    assert dmr.grouped_layer_norm(x, off[:1].contiguous()).shape == (0, 8)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("C", [37, 64, 1024, 4200])
def test_norm_unaligned_arrays(dmr, C, dtype):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs([40, 3], C, dtype, 5)
    offd = torch.from_numpy(off).to(DEV)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    y = shifted(torch.zeros_like(x))
    dmr.dmr_grouped_layer_norm_fwd(shifted(x), offd, shifted(w), shifted(b), y)
    _check(y, layer_norm_forward(x64, off, w64, b64), layer_norm_forward_bound(x64, off, w64, b64, dtype), "y")
    for got, ref, bound in zip(_backward(dmr, shifted(x), offd, shifted(w), shifted(g)), layer_norm_backward(x64, off, w64, g64),
                               layer_norm_backward_bound(x64, off, w64, g64, dtype)):
        _check(got, ref, bound, "grad")


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("C", [37, 64, 1024, 4200])
def test_norm_non_finite_values_stay_in_their_row_and_group(dmr, C, dtype):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs([33, 20, 0, 90], C, dtype, 6)
    offd = torch.from_numpy(off).to(DEV)
    x[40, 5], x[2, 0] = float("inf"), float("nan")
    clean = np.ones(len(x64), bool)
    clean[[2, 40]] = False
    y = dmr.grouped_layer_norm(x, offd, w, b).double().cpu().numpy()
    ref, bound = layer_norm_forward(x64, off, w64, b64), layer_norm_forward_bound(x64, off, w64, b64, dtype)
    assert (np.abs(y - ref)[clean] <= bound[clean]).all() and np.isnan(y[~clean]).all()
    gx, gw, gb = (t.double().cpu().numpy() for t in _backward(dmr, x, offd, w, g))
    (rx, rw, rb), (bx, bw, bb) = layer_norm_backward(x64, off, w64, g64), layer_norm_backward_bound(x64, off, w64, g64, dtype)
    assert (np.abs(gx - rx)[clean] <= bx[clean]).all() and np.isnan(gx[~clean]).all()
    assert np.isnan(gw[:2]).all() and (np.abs(gw - rw)[2:] <= bw[2:]).all() and (np.abs(gb - rb) <= bb).all()


@pytest.mark.parametrize("C", [60, 64, 5000])
def test_norm_leaves_rows_of_no_group_as_they_are(dmr, C):
    x, g = torch.randn((50, C), device=DEV), torch.randn((50, C), device=DEV)
    off = torch.tensor([0, 20, 30], device=DEV)
    y = torch.full_like(x, 7.0)
    dmr.dmr_grouped_layer_norm_fwd(x, off, None, None, y)
    assert (y[30:] == 7.0).all()
    gx = torch.full_like(x, 7.0)
    dmr.dmr_grouped_layer_norm_bwd(x, off, None, g, gx, None, None)
    assert (gx[30:] == 7.0).all()
    part = dmr.grouped_layer_norm(x[:30].contiguous(), off)
    assert torch.equal(y[:30], part)


def test_norm_results_repeat_and_use_the_current_stream(dmr):
    off, (x, _), (w, _), (b, _), (g, _) = _inputs([40000, 10, 30000], 64, "float32", 7)
    offd = torch.from_numpy(off).to(DEV)
    first = [dmr.grouped_layer_norm(x, offd, w, b)] + _backward(dmr, x, offd, w, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [dmr.grouped_layer_norm(x, offd, w, b)] + _backward(dmr, x, offd, w, g)
    side.synchronize()
    for a, c in zip(first, again):
        assert torch.equal(a, c)


def test_norm_autograd(dmr):
    off, (x, x64), (w, w64), (b, b64), (g, g64) = _inputs([10, 0, 25], 12, "float32", 8)
    offd = torch.from_numpy(off).to(DEV)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    dmr.grouped_layer_norm(leaves[0], offd, leaves[1], leaves[2]).backward(g.t().contiguous().t())   # not contiguous
    for t, r, bound in zip(leaves, layer_norm_backward(x64, off, w64, g64), layer_norm_backward_bound(x64, off, w64, g64, "float32")):
        _check(t.grad, r, bound, "grad")
    w2 = w.clone().requires_grad_(True)
    dmr.grouped_layer_norm(x, offd, w2).backward(g)
    assert torch.equal(w2.grad, leaves[1].grad)
    assert not dmr.grouped_layer_norm(x, offd, w, b).requires_grad
    # second derivatives and forward mode raise
    xg = x.clone().requires_grad_(True)
    (gx,) = torch.autograd.grad(dmr.grouped_layer_norm(xg, offd).square().sum(), xg, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            dmr.grouped_layer_norm(dual, offd)


def test_norm_refusals(dmr):
    x, w = torch.zeros((4, 8), device=DEV), torch.zeros((2, 8), device=DEV)
    off = torch.tensor([0, 1, 4], dtype=torch.int64, device=DEV)
    y = torch.zeros((4, 8), device=DEV)
    for bad in (dict(x=x.half()), dict(x=x.double()), dict(x=x[0]), dict(off=off.int()), dict(off=off[:2].contiguous()),
                dict(w=w[:, :7]), dict(w=w.cpu()), dict(x=torch.zeros((8, 4), device=DEV).t()), dict(y=y[:3]), dict(b=w[0]),
                dict(off=off[0])):
        a = dict(x=x, off=off, w=w, b=None, y=y)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            dmr.dmr_grouped_layer_norm_fwd(a["x"], a["off"], a["w"], a["b"], a["y"])
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(dmr.DmrError):
            dmr.grouped_layer_norm(x, off, w, eps=eps)
    with pytest.raises(TypeError):
        dmr.grouped_layer_norm(x.double(), off)
    with pytest.raises(ValueError):      # the gradient of the weight needs a workspace
        dmr.dmr_grouped_layer_norm_bwd(x, off, w, y, None, torch.empty_like(w), None)
    with pytest.raises(dmr.DmrError):
        dmr.dmr_grouped_layer_norm_bwd(x, off, w, y, None, torch.empty_like(w), None, torch.empty(16, dtype=torch.uint8, device=DEV))


def test_norm_past_32_bit_offsets(dmr):
    for C in (2048, 2047):
        R, tail = (1 << 20) + 3000, 200
        say(f"[gpu] layer norm {R} rows of {C}")
        off = np.array([0, 1 << 20, R - 70, R], np.int64)
        x = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV)
        g = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV)
        rng = np.random.default_rng(1)
        (xt, x64), (gt, g64) = _typed(rng.normal(size=(tail, C)), "bfloat16"), _typed(rng.normal(size=(tail, C)), "bfloat16")
        x[R - tail:], g[R - tail:] = xt, gt
        w, w64 = _typed(rng.normal(size=(3, C)), "bfloat16")
        offd = torch.from_numpy(off).to(DEV)
        last = np.array([0, 0, tail - 70, tail], np.int64)
        y = dmr.grouped_layer_norm(x, offd, w)
        _check(y[R - tail:], layer_norm_forward(x64, last, w64), layer_norm_forward_bound(x64, last, w64, None, "bfloat16"), "y")
        assert (y[:R - tail] == 0).all()
        grads = _backward(dmr, x, offd, w, g)
        ref, bound = layer_norm_backward(x64, last, w64, g64), layer_norm_backward_bound(x64, last, w64, g64, "bfloat16")
        _check(grads[0][R - tail:], ref[0], bound[0], "gx")
        for k in (1, 2):
            _check(grads[k], ref[k], bound[k], "gw, gb")
        del x, g, y, grads


# ----------------------------------------------------------------------------


def _check_clip(dmr, shapes, dtypes, groups, max_norm=1.0, seed=0, scale=None, eps=1e-6):
    say(f"[gpu] clip {len(shapes)} tensors, groups {groups}")
    rng = np.random.default_rng(seed)
    count = groups or 1
    values = sum(int(np.prod(s)) for s in shapes) // count
    by = np.exp(rng.normal(size=count)) / max(values, 1) ** 0.5 if scale is None else np.full(count, scale)
    pairs = []
    for s, d in zip(shapes, dtypes):
        a = rng.normal(size=(count, int(np.prod(s)) // count)) * by[:, None]
        pairs.append(_typed(a.reshape(s), d))
    ref, norms = clip_grad_norm([p[1] for p in pairs], max_norm, count, eps)
    for inplace in (False, True):
        grads = [p[0].clone() for p in pairs]
        out, n = dmr.clip_grad_norm(grads, max_norm, groups, eps=eps, out=grads if inplace else None)
        n64 = n.double().cpu().numpy()
        with np.errstate(over="ignore"):
            assert (np.abs(n64 - norms) <= 1.01 * 2.0 ** -24 * norms + 2.0 ** -149).all()
        clipped = norms + eps > max_norm
        for o, g, r, d, p in zip(out, grads, ref, dtypes, pairs):
            assert (o is g) == inplace and o.shape == g.shape and o.dtype == g.dtype
            _check(o, r, clip_bound(r, d), "clipped")
            if not inplace:
                assert torch.equal(g, p[0])
            keep = torch.from_numpy(~clipped).to(DEV)
            assert torch.equal(o.reshape(count, -1)[keep], p[0].reshape(count, -1)[keep])   # a factor of 1
    return norms


# small groups (a workgroup each) and large ones, sizes that end inside a
# vector and a chunk, and slices that start anywhere
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("groups,sizes", [(4, [1]), (4, [3, 64, 1, 7]), (16, [64 * 64, 64, 3 * 64]), (3, [21845, 1]), (3, [65536]),
                                          (2, [65537]), (3, [8191, 70001, 5]), (1, [100003]), (2, [400000, 8192, 16384]),
                                          (300, [33, 2]), (5, [0, 10]), (5, [0])])
def test_clip_per_group(dmr, groups, sizes, dtype):
    _check_clip(dmr, [(groups, s) for s in sizes], [dtype] * len(sizes), groups)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("shapes", [[(1,)], [(7, 3), (5,)], [()], [(16, 64, 64), (16, 64)], [(300, 1000), (0, 5), (17,)],
                                    [(1 << 20,), (999,), (3, 5, 7)]])
@pytest.mark.parametrize("max_norm", [0.1, 1e6, 0.0])
def test_clip_all_together(dmr, shapes, max_norm, dtype):
    _check_clip(dmr, shapes, [dtype] * len(shapes), None, max_norm)


def test_clip_of_mixed_types_and_of_more_tensors_than_a_launch_takes(dmr):
    kinds = list(TORCH)
    for sizes, groups in (([100] * 150, 3), ([3000] * 150, 2), ([70000] * 2 + [5] * 128 + [40000], None)):
        _check_clip(dmr, [(groups or 1, s) for s in sizes], [kinds[k % 3] for k in range(len(sizes))], groups)


def test_clip_of_very_small_and_large_values(dmr):
    # squares pass float32's range at both ends, the norms do not
    for scale in (1e-30, 1e30):
        _check_clip(dmr, [(2, 5000), (2, 9)], ["float32"] * 2, 2, max_norm=scale, scale=scale, eps=0.0)
        _check_clip(dmr, [(2, 90000), (2, 9)], ["float32"] * 2, 2, max_norm=scale, scale=scale, eps=0.0)
    # a norm past float32's range itself: infinite as it is stored, but the values are scaled by it
    big = torch.full((4,), 3e38, device=DEV)
    (out,), n = dmr.clip_grad_norm([big], 1.0)
    assert torch.isinf(n).all() and torch.allclose(out, torch.full_like(out, 0.5))


@pytest.mark.parametrize("size", [50, 70000])
def test_clip_of_non_finite_values_touches_no_other_group(dmr, size):
    g = torch.randn((4, size), device=DEV)
    h = torch.randn((4, 9), device=DEV).half()
    clean, _ = dmr.clip_grad_norm([g, h], 1.0, groups=4)
    g[1, 17], h[2, 3] = float("inf"), float("nan")
    out, n = dmr.clip_grad_norm([g, h], 1.0, groups=4)
    assert torch.isinf(n[1]) and torch.isnan(n[2]) and torch.isfinite(n[[0, 3]]).all()
    for o, c in zip(out, clean):
        assert torch.equal(o[[0, 3]], c[[0, 3]]) and torch.isnan(o[2]).all()
    assert torch.isnan(out[0][1, 17]) and (out[0][1, :17] == 0).all() and (out[1][1] == 0).all()


def test_clip_of_zeros(dmr):
    for eps in (1e-6, 0.0):
        (out,), n = dmr.clip_grad_norm([torch.zeros(1000, device=DEV)], 0.5, eps=eps)
        assert (out == 0).all() and (n == 0).all()


def test_clip_past_32_bit_offsets(dmr):
    # two groups of more than 2^32 bytes; the second's values lie past it
    g = torch.zeros((2, (1 << 31) + 5), dtype=torch.bfloat16, device=DEV)
    g[0, -1], g[1, 0], g[1, -1] = 3.0, 6.0, 8.0
    (out,), n = dmr.clip_grad_norm([g], 5.0, groups=2)
    assert n.tolist() == [3.0, 10.0]
    assert out[0, -1] == 3.0 and out[1, 0] == 3.0 and out[1, -1] == 4.0 and out.count_nonzero() == 3


def test_clip_in_place_is_seen_by_autograd(dmr):
    # a saved tensor that clipping in place has changed is not differentiated with
    w = torch.randn(10, device=DEV, requires_grad=True)
    v = torch.randn(10, device=DEV)
    loss = (w * v).sum()
    dmr.clip_grad_norm([v], 0.1, out=[v])
    with pytest.raises(RuntimeError):
        loss.backward()


def test_clip_streams_and_refusals(dmr):
    grads = [torch.randn((3, 50000), device=DEV), torch.randn((3, 7), device=DEV)]
    first, n = dmr.clip_grad_norm(grads, 1.0, groups=3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again, m = dmr.clip_grad_norm(grads, 1.0, groups=3)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first + [n], again + [m]))
    for bad, kw in (([], {}), (grads, dict(groups=2)), (grads, dict(groups=-3)), ([grads[0].t()], {}), ([grads[0].double()], {}),
                    ([grads[0], grads[1].cpu()], {}), (grads, dict(out=grads[:1])), (grads, dict(out=[grads[0], grads[0]])),
                    (grads, dict(out=[g.half() for g in grads])), ([torch.tensor(1.0, device=DEV)], dict(groups=1))):
        with pytest.raises((TypeError, ValueError)):
            dmr.clip_grad_norm(bad, 1.0, **kw)
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=-1.0)):
        with pytest.raises(dmr.DmrError):
            dmr.clip_grad_norm(grads, **kw)
    norms = torch.empty(3, device=DEV)
    with pytest.raises(dmr.DmrError):
        dmr.dmr_clip_norm([torch.zeros((3, 90000), device=DEV)] * 1, [torch.zeros((3, 90000), device=DEV)], norms, None, 1.0, 3)
    with pytest.raises(ValueError):
        dmr.dmr_clip_norm(grads, grads, norms[:2], None, 1.0, 3)


def test_norms_and_clipping_in_a_graph(dmr):
    off = torch.tensor([0, 300, 300, 20000], dtype=torch.int64, device=DEV)
    x, w, g = torch.randn(20000, 64, device=DEV), torch.randn(3, 64, device=DEV), torch.randn(20000, 64, device=DEV)
    small, large = torch.randn(3, 500, device=DEV), torch.randn(3, 90000, device=DEV)

    def work():
        y = dmr.grouped_layer_norm(x, off, w)
        grads = _backward(dmr, x, off, w, g)
        one, n = dmr.clip_grad_norm([grads[1], small], 1.0, groups=3)
        two, m = dmr.clip_grad_norm([grads[0], large], 1.0)
        return [y, *grads, *one, n, *two, m]

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
        large.copy_(torch.randn_like(large))
        eager = work()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
