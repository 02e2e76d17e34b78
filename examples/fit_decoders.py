"""Fits one small decoder per mesh to depth images, through the rasterizer.

    python examples/fit_decoders.py [--deep]

A batch of spheres of different sizes is bent towards target shapes that are
only seen as depth images. Every mesh has its own two-layer decoder from
features of a vertex to its offset: grouped_linear applies each mesh's weights
to its own packed vertices, project_meshes and rasterize_meshes make the
image, the gradients come back through all of them, and every weight moves by
its orthogonalised momentum (orthogonalize). With --deep a decoder is a block
with a norm and a gated layer (grouped_layer_norm, grouped_gated_linear) before
its head, and each mesh's gradients are clipped by their own norm
(clip_grad_norm).
"""

from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import differentiable_mesh_rasterization_amd as dmr  # noqa: E402
from workloads.meshes import icosphere  # noqa: E402

WIDTH = 64


def spheres(levels, device):
    """Packed icospheres: positions [V, 3], faces [F, 3], vertex and face offsets."""
    verts, faces, vo, fo = [], [], [0], [0]
    for level in levels:
        v, f = icosphere(level)
        verts.append(v)
        faces.append(f + vo[-1])
        vo.append(vo[-1] + len(v))
        fo.append(fo[-1] + len(f))
    return (torch.from_numpy(np.concatenate(verts).astype(np.float32)).to(device),
            torch.from_numpy(np.concatenate(faces)).to(device),
            torch.tensor(vo, dtype=torch.int64, device=device), torch.tensor(fo, dtype=torch.int64, device=device))


def cameras(count, device):
    """One pinhole camera per mesh, two units in front of the unit sphere's centre."""
    m = torch.zeros((count, 4, 4), device=device)
    m[:, 0, 0] = m[:, 1, 1] = 1.6
    m[:, 2, 2] = m[:, 3, 2] = 1.0
    m[:, 2, 3] = m[:, 3, 3] = 2.0
    return m


class Decoders:
    """offset = W2 relu(W1 features + b1), one (W1, b1, W2) per mesh."""

    def __init__(self, count, device, seed=0):
        gen = torch.Generator(device="cpu").manual_seed(seed)
        self.w1 = (torch.randn((count, WIDTH, WIDTH), generator=gen) / WIDTH ** 0.5).to(device).requires_grad_(True)
        self.b1 = torch.zeros((count, WIDTH), device=device, requires_grad=True)
        self.w2 = torch.zeros((count, 3, WIDTH), device=device, requires_grad=True)
        self.momentum = [torch.zeros_like(w) for w in (self.w1, self.w2)]

    def __call__(self, features, offsets):
        hidden = torch.relu(dmr.grouped_linear(features, offsets, self.w1, self.b1))
        return dmr.grouped_linear(hidden, offsets, self.w2)

    @torch.no_grad()
    def step(self, rate, keep=0.9):
        """Momentum, orthogonalised: every matrix moves by `rate` in each of its directions."""
        for w, mom in zip((self.w1, self.w2), self.momentum):
            mom.mul_(keep).add_(w.grad)
            w -= rate * dmr.orthogonalize(mom)
            w.grad = None
        self.b1 -= rate * torch.nn.functional.normalize(self.b1.grad, dim=1)
        self.b1.grad = None


class DeepDecoders:
    """offset = W3 (h + W2 gated(norm(h))), h = W1 features + b1, one of each weight per mesh."""

    def __init__(self, count, device, seed=0, hidden=2 * WIDTH):
        gen = torch.Generator(device="cpu").manual_seed(seed)

        def weight(*shape):
            return (torch.randn((count, *shape), generator=gen) / shape[-1] ** 0.5).to(device).requires_grad_(True)

        def vector(*shape, value=0.0):
            return torch.full((count, *shape), value, device=device, requires_grad=True)

        self.w1, self.b1 = weight(WIDTH, WIDTH), vector(WIDTH)
        self.gamma, self.beta = vector(WIDTH, value=1.0), vector(WIDTH)
        self.gate, self.gate_bias = weight(2, hidden, WIDTH), vector(2, hidden)
        self.w2, self.w3 = weight(WIDTH, hidden), vector(3, WIDTH)
        self.matrices = [self.w1, self.gate, self.w2, self.w3]
        self.vectors = [self.b1, self.gamma, self.beta, self.gate_bias]
        self.momentum = [torch.zeros_like(w) for w in self.matrices]

    def __call__(self, features, offsets):
        h = dmr.grouped_linear(features, offsets, self.w1, self.b1)
        inner = dmr.grouped_layer_norm(h, offsets, self.gamma, self.beta)
        inner = dmr.grouped_gated_linear(inner, offsets, self.gate, self.gate_bias)
        return dmr.grouped_linear(h + dmr.grouped_linear(inner, offsets, self.w2), offsets, self.w3)

    @torch.no_grad()
    def step(self, rate, keep=0.9, max_norm=1.0):
        """Each mesh's gradients clipped to max_norm, then momentum, orthogonalised, for the matrices."""
        everything = self.matrices + self.vectors
        grads = [p.grad for p in everything]
        dmr.clip_grad_norm(grads, max_norm, groups=len(self.w1), out=grads)
        for w, mom in zip(self.matrices, self.momentum):
            mom.mul_(keep).add_(w.grad)
            planes = mom.view(-1, *mom.shape[-2:])
            w -= rate * dmr.orthogonalize(planes).view(w.shape)
        for v in self.vectors:
            v -= rate * torch.nn.functional.normalize(v.grad.flatten(1), dim=1).view(v.shape)
        for p in everything:
            p.grad = None


def depth_images(world, faces, vert_offsets, face_offsets, cams, side):
    screen = dmr.project_meshes(world, vert_offsets, cams)
    p2f, zbuf, _, _ = dmr.rasterize_meshes(screen, faces, face_offsets, (side, side))
    return p2f[..., 0] >= 0, zbuf[..., 0]


def fit(steps=40, levels=(2, 4, 3, 1), side=64, rate=0.02, device="cuda:0", report=None, deep=False):
    """The mean squared depth error of every step."""
    device = torch.device(device)
    base, faces, vo, fo = spheres(levels, device)
    cams = cameras(len(levels), device)
    waves = torch.from_numpy(np.random.default_rng(1).normal(0.0, 2.0, (3, WIDTH)).astype(np.float32)).to(device)
    features = torch.sin(base @ waves)
    target = base * (1.0 + 0.2 * torch.sin(3.0 * base[:, :1]) * torch.cos(2.0 * base[:, 1:2]))
    seen, depth = depth_images(target, faces, vo, fo, cams, side)
    decoders, losses = (DeepDecoders if deep else Decoders)(len(levels), device), []
    for k in range(steps):
        covered, z = depth_images(base + decoders(features, vo), faces, vo, fo, cams, side)
        both = (covered & seen).float()
        loss = (both * (z - depth) ** 2).sum() / both.sum()
        loss.backward()
        decoders.step(rate * (1.0 - k / steps))
        losses.append(float(loss.detach()))
        if report:
            report(k, losses[-1])
    return losses


if __name__ == "__main__":
    fit(deep="--deep" in sys.argv, report=lambda k, loss: print(f"step {k:3d}  depth error {loss:.6f}", flush=True))
