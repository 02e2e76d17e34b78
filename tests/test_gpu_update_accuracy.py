"""The orthogonalised updates on the GPU where their arithmetic is hardest.

Tolerance: X and the factors of the products hold at least 22 bits where
float32 holds 24, so the result may be off by four times what the same
iteration in float32 is off by (oracle/orthogonalize.py: float32_error), plus
its rounding to the output's type (the exact result's own rounding error, and
a twentieth more, since the values that are rounded differ a little)."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say
from oracle.orthogonalize import float32_error, orthogonalize

pytestmark = pytest.mark.gpu

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _typed(a, dtype):
    """(device tensor of the type, the values it holds in float64)"""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


def _rounding(ref, dtype):
    return float(np.linalg.norm(torch.from_numpy(ref).to(TORCH[dtype]).to(torch.float64).numpy() - ref))


def check_update(got, u64, dtype, steps=5, eps=1e-7):
    got = got.to(torch.float64).cpu().numpy()
    assert got.shape == u64.shape
    for k in range(len(u64)):
        ref = orthogonalize(u64[k], steps, eps)
        bound = 1.05 * _rounding(ref, dtype) + 4 * float32_error(u64[k], steps, eps)
        err = np.linalg.norm(got[k] - ref)
        assert err <= bound, (k, err / bound, err / np.linalg.norm(ref))    # a NaN fails too


# a momentum of few strong directions: the weak ones are stretched most, and
# with them what the products of the strong ones lose
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("m,n,rank,noise", [(60, 60, 8, 1e-3), (256, 256, 32, 1e-3), (300, 130, 16, 1e-2), (512, 600, 64, 1e-3)])
def test_update_of_few_strong_directions(dmr, m, n, rank, noise, dtype):
    say(f"[gpu] orthogonalize {dtype} {m}x{n} rank {rank}")
    rng = np.random.default_rng(rank)
    strong = rng.normal(size=(2, m, rank)) @ rng.normal(size=(2, rank, n)) / np.sqrt(rank)
    u, u64 = _typed(1e-2 * (strong + noise * rng.normal(size=(2, m, n))), dtype)
    check_update(dmr.orthogonalize(u), u64, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n", [(64, 64), (100, 260)])
@pytest.mark.parametrize("top", [1e37, 3e38])
def test_update_whose_norm_passes_float32(dmr, m, n, top, dtype):
    u, u64 = _typed(np.random.default_rng(4).uniform(-top, top, size=(2, m, n)), dtype)
    assert np.isfinite(u64).all() and np.linalg.norm(u64[0]) > 3.5e38
    check_update(dmr.orthogonalize(u), u64, dtype)


@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("m,n", [(8, 12), (100, 260)])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -126, 1e-30])
def test_update_of_zeros_for_any_eps(dmr, m, n, eps, dtype):
    u = torch.zeros((2, m, n), dtype=TORCH[dtype], device=DEV)
    for steps in (1, 5):
        assert (dmr.orthogonalize(u, steps, eps) == 0).all()


# |U| and eps both far below 1, down to float32's subnormal values
@pytest.mark.parametrize("m,n", [(8, 12), (100, 260)])
@pytest.mark.parametrize("norm,eps", [(1e-36, 1e-12), (1e-36, 1e-38), (1e-38, 2.0 ** -126), (1e-40, 2.0 ** -140)])
@pytest.mark.parametrize("steps", [1, 5])
def test_update_of_tiny_values(dmr, m, n, norm, eps, steps):
    eps = float(np.float32(eps))
    u, u64 = _typed(np.random.default_rng(6).normal(size=(1, m, n)) * norm / np.sqrt(m * n), "float32")
    check_update(dmr.orthogonalize(u, steps, eps), u64, "float32", steps, eps)


# |U| = t eps: X starts at t and grows by 3.4445 a step at most
@pytest.mark.parametrize("dtype", list(TORCH))
@pytest.mark.parametrize("m,n", [(40, 30), (96, 200), (150, 90)])
@pytest.mark.parametrize("t,steps", [(1e-25, 5), (1e-6, 8), (1e-8, 12), (1e-10, 16), (1e-9, 20), (1e-33, 64)])
def test_update_far_below_eps(dmr, m, n, t, steps, dtype):
    say(f"[gpu] orthogonalize {dtype} {m}x{n} at {t} of eps, {steps} steps")
    u, u64 = _typed(np.random.default_rng(steps).normal(size=(2, m, n)) * 1e-2, dtype)
    eps = float(np.float32(np.linalg.norm(u64[0]) / t))
    check_update(dmr.orthogonalize(u, steps, eps), u64, dtype, steps, eps)


@pytest.mark.parametrize("m,n", [(40, 30), (150, 90)])
def test_update_of_matrices_of_different_norms(dmr, m, n):
    u, u64 = _typed(np.random.default_rng(3).normal(size=(4, m, n)) * np.array([1.0, 1e-13, 1e-7, 1e-30])[:, None, None], "float32")
    check_update(dmr.orthogonalize(u, 10), u64, "float32", 10)


@pytest.mark.parametrize("m,n", [(8, 12), (100, 260)])
@pytest.mark.parametrize("steps", [1, 5, 40, 64])
def test_update_of_subnormal_values_far_below_eps(dmr, m, n, steps):
    u, u64 = _typed(np.random.default_rng(7).normal(size=(1, m, n)) * 3e-43, "float32")
    check_update(dmr.orthogonalize(u, steps, 1.0), u64, "float32", steps, 1.0)


@pytest.mark.parametrize("m,n", [(1, 1), (3, 64), (8, 12), (40, 30), (64, 400), (100, 260)])
@pytest.mark.parametrize("norm,eps,steps", [(1e-40, 1.0, 40), (1e-30, 1e13, 40), (1e-2, 1e38, 25), (1e-43, 1e-3, 64)])
def test_update_below_float32_of_eps_is_linear(dmr, m, n, norm, eps, steps):
    # X_0 itself is below float32's normal values, the result, 3.4445^steps X_0, is not: a step rounds X to
    # 22 bits or more and adds float32 values, 2^-20 together
    eps = float(np.float32(eps))
    u, u64 = _typed(np.random.default_rng(8).normal(size=(2, m, n)) * norm / np.sqrt(m * n), "float32")
    got = dmr.orthogonalize(u, steps, eps).to(torch.float64).cpu().numpy()
    ref = orthogonalize(u64, steps, eps)
    for g, r in zip(got, ref):
        assert np.linalg.norm(g - r) <= steps * 2.0 ** -20 * np.linalg.norm(r)
