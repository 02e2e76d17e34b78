"""Norm, gated layer, linear layer, clipping and orthogonalised updates
together, as one block of a decoder per mesh is trained: its gradients against
the same block in float64 on the CPU, a whole step captured in a graph, and the
example that is made of them.

Tolerance of the float32 gradients, in the 2-norm: ten stages forward and back,
sums of at most 64 terms each off by 64 2^-23 of the sum of magnitudes, which
is at most 16 times the sum's size for these random values: 10 * 64 * 16 * 2^-23
= 1.2e-3."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, say

pytestmark = pytest.mark.gpu

TOLERANCE = 10 * 64 * 16 * 2.0 ** -23


@pytest.fixture(scope="module")
def dmr():
    return require_gpu()


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fit_decoders.py")
    spec = importlib.util.spec_from_file_location("fit_decoders", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def _block(dmr, x, off, p):
    inner = dmr.grouped_layer_norm(x, off, p["gamma"], p["beta"])
    inner = dmr.grouped_gated_linear(inner, off, p["gate"], p["gate_bias"], "gelu")
    return x + dmr.grouped_linear(inner, off, p["down"], p["down_bias"])


def _reference(x, off, p):
    rows = []
    for n, (a, b) in enumerate(zip(off, off[1:])):
        v = x[a:b]
        h = (v - v.mean(dim=1, keepdim=True)) / torch.sqrt(v.var(dim=1, correction=0, keepdim=True) + 1e-5)
        h = h * p["gamma"][n] + p["beta"][n]
        gate, up = (h @ p["gate"][n][k].T + p["gate_bias"][n][k] for k in (0, 1))
        act = gate * 0.5 * torch.erfc(-gate / 2 ** 0.5)
        rows.append(v + (act * up) @ p["down"][n].T + p["down_bias"][n])
    return torch.cat(rows)


def _parameters(N, C, F, seed=0):
    rng = np.random.default_rng(seed)
    shapes = dict(gamma=(N, C), beta=(N, C), gate=(N, 2, F, C), gate_bias=(N, 2, F), down=(N, C, F), down_bias=(N, C))
    return {k: torch.from_numpy(rng.normal(size=s) / (s[-1] ** 0.5 if len(s) > 2 else 1.0) + (k == "gamma")).float()
            for k, s in shapes.items()}


@pytest.mark.parametrize("sizes,C,F", [([30, 0, 1, 69], 16, 24), ([200, 3, 150], 37, 64), ([40, 60], 64, 50)])
def test_gradients_of_a_block(dmr, sizes, C, F):
    say(f"[gpu] block {C} {F} sizes {sizes}")
    off = np.concatenate([[0], np.cumsum(sizes)])
    rng = np.random.default_rng(1)
    x, g = (torch.from_numpy(rng.normal(size=(off[-1], C))).float() for _ in range(2))
    p = _parameters(len(sizes), C, F)
    leaves = {k: v.to(DEV).requires_grad_(True) for k, v in dict(p, x=x).items()}
    y = _block(dmr, leaves["x"], torch.from_numpy(off).to(DEV), leaves)
    y.backward(g.to(DEV))
    exact = {k: v.double().requires_grad_(True) for k, v in dict(p, x=x).items()}
    ref = _reference(exact["x"], off, exact)
    ref.backward(g.double())
    pairs = {"y": (y.detach(), ref.detach()), **{k: (leaves[k].grad, exact[k].grad) for k in exact}}
    for k, (got, want) in pairs.items():
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= TOLERANCE, (k, err)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_training_step_in_a_graph(dmr, dtype):
    # forward, backward, clipping per mesh and in place, and the update, replayed
    off = torch.tensor([0, 500, 500, 3000], device=DEV)
    p = {k: v.to(DEV).to(dtype) for k, v in _parameters(3, 64, 96).items()}
    x, g = torch.randn((3000, 64), device=DEV).to(dtype), torch.randn((3000, 64), device=DEV).to(dtype)

    def work():
        leaves = {k: v.detach().requires_grad_(True) for k, v in p.items()}
        grads = list(torch.autograd.grad(_block(dmr, x, off, leaves), list(leaves.values()), g))
        clipped, norms = dmr.clip_grad_norm(grads, 1.0, groups=3, out=grads)
        return [*clipped, norms, dmr.orthogonalize(clipped[2].view(6, 96, 64))]

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
        assert (out[6] > 1.0).any()      # something was clipped


def test_two_streams_at_once(dmr):
    # calls that share inputs, on two streams, each with workspaces of its own
    off = torch.tensor([0, 20000, 50000], device=DEV)
    p = {k: v.to(DEV) for k, v in _parameters(2, 64, 128).items()}
    x, g = torch.randn((50000, 64), device=DEV), torch.randn((50000, 64), device=DEV)

    def work():
        leaves = {k: v.detach().requires_grad_(True) for k, v in p.items()}
        grads = torch.autograd.grad(_block(dmr, x, off, leaves), list(leaves.values()), g)
        return [*grads, *dmr.clip_grad_norm(grads, 1.0)[0]]

    alone = work()
    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            results.append([work() for _ in range(3)])
    torch.cuda.synchronize()
    for runs in results:
        for r in runs:
            for a, b in zip(alone, r):
                assert torch.equal(a, b)


def test_deep_decoders_run_and_their_gradients_reach_every_weight(dmr):
    example = _example()
    say("[gpu] fit 4 deep decoders, 3 steps")
    losses = example.fit(steps=3, deep=True)
    assert len(losses) == 3 and np.isfinite(losses).all()
    # the head starts at zero: one step moves it, and then every weight has a gradient
    device = torch.device(DEV)
    decoders = example.DeepDecoders(2, device)
    off = torch.tensor([0, 40, 100], device=device)
    features, target = torch.randn((100, example.WIDTH), device=device), torch.randn((100, 3), device=device)
    for k in range(2):
        before = [w.detach().clone() for w in decoders.matrices]
        (decoders(features, off) - target).square().mean().backward()
        grads = [w.grad.clone() for w in decoders.matrices + decoders.vectors]
        decoders.step(0.01)
    for w, b, gr in zip(decoders.matrices, before, grads):
        assert torch.isfinite(gr).all() and (gr != 0).any() and (w.detach() != b).any()
    assert all((v != 0).any() for v in grads)
