"""What the gated layers' backward pass holds between its products, in 16-bit
types: [da du] with float32's range and more bits than the type has, in each
form of the pass.

Tolerances: as in test_gpu_gated.py (oracle/grouped_gated.py)."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from test_gpu_gated import _backward, _check, _typed
from oracle.grouped_gated import gated_backward, gated_backward_bound

pytestmark = pytest.mark.gpu

# one kernel of both widths; one row for each of many groups; the linear layer's
# kernels with small tiles, with the largest ones, and unaligned
FORMS = [([3000, 0, 5], 64, 64), ([3000, 0, 5], 37, 100), ([1] * 64, 136, 300), ([500, 30], 136, 72),
         ([9000, 8000], 1024, 520), ([2000, 3], 131, 77)]


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _type(dtype):
    return getattr(torch, dtype)


def _check_in_range(got, ref, bound, dtype):
    most = torch.finfo(_type(dtype)).max
    for v, r, e, what in zip(got, ref, bound, ("gx", "gw", "gb")):
        past = np.abs(r) - e > 1.001 * most      # of the type's range: rounded to infinity
        assert (v.double().cpu().numpy()[past] == np.sign(r[past]) * np.inf).all(), what
        near = (np.abs(r) + e > most) & ~past
        _check(torch.where(torch.from_numpy(past | near).to(DEV), 0, v), np.where(past | near, 0.0, r), e, what)


def _run(dmr, sizes, cin, cout, dtype, x, w, b, g):
    say(f"[gpu] gated precision {dtype} {cin}->{cout} sizes {sizes[:4]}")
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    (x, x64), (w, w64), (b, b64), (g, g64) = (_typed(v, dtype) for v in (x, w, b, g))
    got = _backward(dmr, x, torch.from_numpy(off).to(DEV), w, b, g)
    ref, bound = (f(x64, off, w64, b64, g64, *rest) for f, rest in ((gated_backward, ()), (gated_backward_bound, (dtype,))))
    _check_in_range(got, ref, bound, dtype)
    return ref


def _shapes(sizes, cin, cout, seed):
    rng = np.random.default_rng(seed)
    R, N = sum(sizes), len(sizes)
    return rng.normal(size=(R, cin)), rng.normal(size=(N, 2, cout, cin)) / cin ** 0.5, 0.3 * rng.normal(size=(N, 2, cout)), \
        rng.normal(size=(R, cout))


@pytest.mark.parametrize("sizes,cin,cout", FORMS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gradients_are_rounded_once(dmr, sizes, cin, cout, dtype):
    # values of one sign, which do not average the roundings of [da du] out: u,
    # act(a) and act'(a) are about 1, and 1 + 1/3 of a step of the type remain
    step = 2.0 ** -10 if dtype == "float16" else 2.0 ** -7
    x, w, b, g = _shapes(sizes, cin, cout, 0)
    x, w, g = np.abs(x), 0.0 * w, np.full_like(g, 1.0 + step)
    b = np.full_like(b, 1.0 + step)
    _run(dmr, sizes, cin, cout, dtype, x, w, b, g)


@pytest.mark.parametrize("sizes,cin,cout", FORMS)
def test_small_float16_gradients_do_not_vanish(dmr, sizes, cin, cout):
    # upstream gradients of 1 to 4 of float16's smallest steps, as a mean over
    # many rows gives them: g u act'(a) is below half a step for most
    x, w, b, g = _shapes(sizes, cin, cout, 1)
    g = 2.0 ** -24 * np.random.default_rng(2).integers(1, 5, size=g.shape)
    _, gw, gb = _run(dmr, sizes, cin, cout, "float16", np.abs(x) + 8.0, w, 0.1 * np.abs(b), g)
    if max(sizes) > 1000:
        assert np.abs(gw).max() > 1000 * 2.0 ** -24


@pytest.mark.parametrize("sizes,cin,cout", FORMS)
def test_large_float16_products_do_not_overflow(dmr, sizes, cin, cout):
    # g u act'(a) of about 100000 with small weights and inputs: every gradient
    # but the bias' first one is inside float16's range
    x, w, b, g = _shapes(sizes, cin, cout, 3)
    b[:, 0], b[:, 1] = 3.0, 400.0
    g = np.where(np.arange(len(g))[:, None] % 97 == 0, 250.0 * np.sign(g), 0.0)
    ref = _run(dmr, sizes, cin, cout, "float16", 2.0 ** -10 * x, 2.0 ** -6 * w, b, g)
    assert np.abs(ref[0]).max() < 60000 and np.abs(ref[1]).max() < 60000


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("sizes,cin,cout", FORMS)
def test_infinite_products_stay_where_they_are(dmr, sizes, cin, cout, dtype):
    # an infinity of [da du] has no low part (it would be NaN); with float16
    # operands, whose low parts may be zero, it gives NaN
    x, w, b, g = _shapes(sizes, cin, cout, 4)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    g[0, 0] = 0.0
    (x, x64), (w, w64), (b, b64), (g, g64) = (_typed(v, dtype) for v in (np.abs(x) + 0.5, np.abs(w) + 0.1, np.abs(b), np.abs(g)))
    ref, bound = gated_backward(x64, off, w64, b64, g64), gated_backward_bound(x64, off, w64, b64, g64, dtype)
    g[0, 0] = float("inf")
    gx, gw, gb = _backward(dmr, x, torch.from_numpy(off).to(DEV), w, b, g)
    if dtype == "bfloat16":
        assert (gx[0] == float("inf")).all() and (gw[0, :, 0] == float("inf")).all()
    assert not torch.isfinite(gx[0]).any() and not torch.isfinite(gw[0, :, 0]).any() and (gb[0, :, 0] == float("inf")).all()
    # the others are as without it
    for v, r, e, at in ((gx, ref[0], bound[0], np.s_[0]), (gw, ref[1], bound[1], np.s_[0, :, 0]), (gb, ref[2], bound[2], np.s_[0, :, 0])):
        v[at], r[at], e[at] = 0.0, 0.0, 1.0
    _check_in_range((gx, gw, gb), ref, bound, dtype)
