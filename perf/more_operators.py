"""What a deeper decoder per mesh needs beside its linear layers: what the operators compute, and on what sizes they are measured.

On packed batches (rows of all groups one after another, row_offsets [N + 1]: group n owns rows
[row_offsets[n], row_offsets[n + 1])):

  grouped_layer_norm    h_r = (x_r - mean x_r) / sqrt(var x_r + eps), y_r = gamma_n h_r + beta_n for every row r of group
                        n, and its backward pass (with the sums over a group's rows for gamma_n and beta_n).
  grouped_gated_linear  y_r = act(A_n x_r + a_n) * (U_n x_r + u_n), weight [N, 2, out, in] = (A, U), bias [N, 2, out] =
                        (a, u), and its backward pass from x, weight, bias and grad_y (nothing else is kept of the
                        forward pass, so both projections are computed again).
  clip_grad_norm        norm_g = sqrt(sum v^2) over the values of all tensors (or, per group, over every tensor's slice g
                        of its first dimension), each value times min(1, max_norm / (norm_g + 1e-6)).

`run` computes them in their plain form (elementary torch operations in 32 bits) where `own` is false, and through the
library's entry points where it is true.
"""

import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "sigmoid")
NORM_EPS = 1e-5
CLIP_EPS = 1e-6
MAX_NORM = 1.0
GELU = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # One token for each of eight meshes before a decoder's hidden layer: the smallest call, all latency.
        dict(name="norm fwd 8x1 rows 64 f16", op="norm_fwd", dtype="float16", groups=8, layout="one", rows=8, width=64),
        # Features of every pixel of 16 images of 256 x 256: the forward pass of an ordinary shading network.
        dict(name="norm fwd pixels 64 bf16", op="norm_fwd", dtype="bfloat16", groups=16, layout="even", rows=1 << 20, width=64),
        # Training on the vertices of the 16-sphere batch, in the rasterizer's own type.
        dict(name="norm bwd spheres 64 f32", op="norm_bwd", dtype="float32", groups=16, layout="levels", rows=217632, width=64),
        # Training wide decoders over ragged groups.
        dict(name="norm bwd ragged 1024 bf16", op="norm_bwd", dtype="bfloat16", groups=32, layout="ragged", rows=65536, width=1024),
        # One query row for each of 64 groups against wide weights, as an autoregressive head calls it: weights are streamed.
        dict(name="gated fwd 64x1 rows 1024-1024 bf16", op="gated_fwd", dtype="bfloat16", groups=64, layout="one", rows=64,
             width=1024, hidden=1024, activation="silu"),
        # A wide block over ragged groups, hidden four times as wide: the largest forward pass.
        dict(name="gated fwd ragged 1024-4096 bf16", op="gated_fwd", dtype="bfloat16", groups=32, layout="ragged", rows=65536,
             width=1024, hidden=4096, activation="silu"),
        # Odd widths, a few short groups and empty ones: nothing is aligned.
        dict(name="gated bwd odd 37-53 f16", op="gated_bwd", dtype="float16", groups=7, layout="ragged", rows=1003, width=37,
             hidden=53, activation="gelu"),
        # Training the shading block of every pixel of 16 images.
        dict(name="gated bwd pixels 64-64 bf16", op="gated_bwd", dtype="bfloat16", groups=16, layout="even", rows=1 << 20,
             width=64, hidden=64, activation="gelu_tanh"),
        # Training the vertex decoder's block on the 16-sphere batch, in the rasterizer's own type.
        dict(name="gated bwd spheres 64-128 f32", op="gated_bwd", dtype="float32", groups=16, layout="levels", rows=217632,
             width=64, hidden=128, activation="silu"),
        # Training wide blocks over ragged groups: the largest call.
        dict(name="gated bwd ragged 1024-4096 bf16", op="gated_bwd", dtype="bfloat16", groups=32, layout="ragged", rows=32768,
             width=1024, hidden=4096, activation="silu"),
        # The gradients of 16 two-block vertex decoders, each mesh with a norm of its own: small tensors.
        dict(name="clip 16 decoders 64-128 f32", op="clip", dtype="float32", groups=16, blocks=2, width=64, hidden=128,
             per_group=True),
        # One norm over the gradients of eight wide two-block decoders.
        dict(name="clip 8 decoders 1024-4096 bf16", op="clip", dtype="bfloat16", groups=8, blocks=2, width=1024, hidden=4096,
             per_group=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _rows(rng, most):
    """groups, layout and rows of a drawn batch of at most `most` rows"""
    groups, layout = _log_uniform(rng, 1, 128), rng.choice(["one", "even", "ragged", "ragged", "levels"])
    if layout == "one":
        groups = min(groups, most)
        return dict(groups=groups, layout=layout, rows=groups)
    if layout == "levels":
        groups = rng.randint(1, 16)
        while groups > 1 and _levels_total(groups) > most:
            groups -= 1
        if _levels_total(groups) <= most:
            return dict(groups=groups, layout=layout, rows=_levels_total(groups))
        layout = "even"
    rows = _log_uniform(rng, 1, max(1, most))
    if layout == "even":
        groups = min(groups, rows)
        rows = rows // groups * groups
    return dict(groups=groups, layout=layout, rows=rows)


def draw(rng):
    dtype, kind = rng.choice(list(DTYPES)), rng.random()
    if kind < 0.2:
        width, hidden, groups = _log_uniform(rng, 3, 1024), _log_uniform(rng, 3, 4096), _log_uniform(rng, 1, 128)
        if rng.random() < 0.5:
            width, hidden = (width + 15) // 16 * 16, (hidden + 15) // 16 * 16
        blocks = rng.randint(1, 8)
        while groups > 1 and groups * blocks * width * hidden > 1 << 26:
            groups //= 2
        while blocks > 1 and groups * blocks * width * hidden > 1 << 26:
            blocks -= 1
        return dict(op="clip", dtype=rng.choice([dtype, "mixed"]), groups=groups, blocks=blocks, width=width, hidden=hidden,
                    per_group=rng.random() < 0.5)
    width = _log_uniform(rng, 3, 2048)
    if rng.random() < 0.5:
        width = (width + 15) // 16 * 16
    if kind < 0.5:
        op = rng.choice(["norm_fwd", "norm_bwd"])
        return dict(op=op, dtype=dtype, width=width, **_rows(rng, min(1 << 20, (1 << 27) // width)))
    op, hidden = rng.choice(["gated_fwd", "gated_bwd"]), _log_uniform(rng, 3, 4096)
    if rng.random() < 0.5:
        hidden = (hidden + 15) // 16 * 16
    passes = 1 if op == "gated_fwd" else 3
    most = min(1 << 20, (1 << 37) // (width * hidden * passes), (1 << 26) // (width + hidden))
    return dict(op=op, dtype=dtype, width=width, hidden=hidden, activation=rng.choice(ACTIVATIONS), **_rows(rng, most))


def _levels_total(groups):
    return sum(10 * 4 ** (3 + i % 4) + 2 for i in range(groups))


def _group_sizes(case, seed):
    """Rows of each group: vertices of icospheres of levels 3 to 6 in some order, equal images, one row each, or a
    ragged split (exponential weights, about one group in eight empty) of the same total."""
    rng = random.Random(seed * 7 + 1)
    groups, rows = case["groups"], case["rows"]
    if case["layout"] == "levels":
        sizes = [10 * 4 ** (3 + i % 4) + 2 for i in range(groups)]
        rng.shuffle(sizes)
        return sizes
    if case["layout"] in ("one", "even"):
        return [rows // groups] * groups
    weights = [0.0 if rng.random() < 0.125 else rng.expovariate(1.0) for _ in range(groups)]
    weights[rng.randrange(groups)] += 0.25
    total, sizes, at, done = sum(weights), [], 0.0, 0
    for w in weights:
        at += w
        upto = min(rows, round(rows * at / total))
        sizes.append(upto - done)
        done = upto
    sizes[max(range(groups), key=lambda g: sizes[g])] += rows - done
    return sizes


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _shapes(case):
    """The tensors of the decoders' blocks: the norm's two, the gated layer's two, the layer back's two."""
    groups, width, hidden = case["groups"], case["width"], case["hidden"]
    block = [(groups, width), (groups, width), (groups, 2, hidden, width), (groups, 2, hidden), (groups, width, hidden),
             (groups, width)]
    return block * case["blocks"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case=case)
    if case["op"] == "clip":
        # gradients of meshes of very different sizes on screen: about half of the norms are above MAX_NORM
        shapes, groups = _shapes(case), case["groups"]
        values = sum(math.prod(s) for s in shapes) // (groups if case["per_group"] else 1)
        scale = torch.exp(_normal((groups,), gen)) * MAX_NORM / math.sqrt(values)
        grads = []
        for s in shapes:
            dtype = DTYPES[case["dtype"]] if case["dtype"] in DTYPES else torch.bfloat16 if len(s) > 2 else torch.float32
            grads.append((_normal(s, gen) * scale.view([groups] + [1] * (len(s) - 1))).to(dtype))
        state["grads"] = grads
        return state
    dtype = DTYPES[case["dtype"]]
    sizes = _group_sizes(case, seed)
    groups, rows, width = case["groups"], case["rows"], case["width"]
    offsets = [0]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    state["longest"] = max(sizes)
    state["row_offsets"] = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    covered = torch.rand((rows, 1), generator=gen, device="cuda") < 0.7  # rows that no pixel sees get no gradient
    if case["op"] in ("norm_fwd", "norm_bwd"):
        # a layer's outputs: rows of different means and scales
        x = _normal((rows, width), gen) * torch.exp(0.5 * _normal((rows, 1), gen)) + 0.5 * _normal((rows, 1), gen)
        state["x"] = x.to(dtype)
        state["weight"] = (1.0 + 0.1 * _normal((groups, width), gen)).to(dtype)
        state["bias"] = (0.1 * _normal((groups, width), gen)).to(dtype)
        if case["op"] == "norm_bwd":
            state["grad_y"] = (_normal((rows, width), gen) * covered).to(dtype)
        return state
    hidden = case["hidden"]
    state["x"] = _normal((rows, width), gen).to(dtype)  # rows after a norm
    state["weight"] = (_normal((groups, 2, hidden, width), gen) / math.sqrt(width)).to(dtype)
    state["bias"] = (0.1 * _normal((groups, 2, hidden), gen)).to(dtype)
    if case["op"] == "gated_bwd":
        state["grad_y"] = (_normal((rows, hidden), gen) * covered).to(dtype)
    return state


def _run_own(s):
    import differentiable_mesh_rasterization_amd as dmr

    op = s["case"]["op"]
    if op == "clip":
        clipped, norms = dmr.clip_grad_norm(s["grads"], MAX_NORM, groups=s["case"]["groups"] if s["case"]["per_group"] else None,
                                            eps=CLIP_EPS)
        return {"grads": clipped, "norms": norms}
    x, row_offsets, weight, bias = s["x"], s["row_offsets"], s["weight"], s["bias"]
    if op == "norm_fwd":
        return dmr.grouped_layer_norm(x, row_offsets, weight, bias, eps=NORM_EPS)
    if op == "gated_fwd":
        return dmr.grouped_gated_linear(x, row_offsets, weight, bias, activation=s["case"]["activation"])
    grads = {"grad_x": torch.empty_like(x), "grad_weight": torch.empty_like(weight), "grad_bias": torch.empty_like(bias)}
    groups = weight.shape[0]
    if op == "norm_bwd":
        size = dmr.dmr_grouped_layer_norm_workspace_size(x.shape[0], groups, x.shape[1], x.dtype)
        workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
        dmr.dmr_grouped_layer_norm_bwd(x, row_offsets, weight, s["grad_y"], workspace=workspace, eps=NORM_EPS, **grads)
        return grads
    size = dmr.dmr_grouped_gated_linear_workspace_size(x.shape[0], groups, x.shape[1], weight.shape[2], x.dtype)
    workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
    dmr.dmr_grouped_gated_linear_bwd(x, row_offsets, weight, bias, s["grad_y"], workspace=workspace,
                                     activation=s["case"]["activation"], **grads)
    return grads


def _slots(s):
    """Each row's group and its place within it, for sums and products over groups padded to the longest."""
    offsets = s["row_offsets"]
    row = torch.arange(s["x"].shape[0], device="cuda")
    group = torch.searchsorted(offsets[1:], row, right=True)
    return group, row - offsets[group]


def _padded(v, s, group, place):
    wide = torch.zeros((s["weight"].shape[0], s["longest"], v.shape[1]), dtype=torch.float32, device="cuda")
    wide[group, place] = v.float()
    return wide


def _activated(a, kind):
    """act(a) and its derivative"""
    if kind == "gelu":
        tail = 0.5 * (1.0 + torch.erf(a / math.sqrt(2.0)))
        return a * tail, tail + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = torch.tanh(GELU * (a + 0.044715 * a**3))
        return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * GELU * (1.0 + 3 * 0.044715 * a * a)
    sig = 1.0 / (1.0 + torch.exp(-a))
    if kind == "silu":
        return a * sig, sig * (1.0 + a * (1.0 - sig))
    return sig, sig * (1.0 - sig)


def _plain_clip(s):
    case, grads = s["case"], s["grads"]
    groups = case["groups"] if case["per_group"] else 1
    squares = [g.float().reshape(groups, -1).square().sum(dim=1) for g in grads]
    norms = torch.stack(squares).sum(dim=0).sqrt()
    scale = (MAX_NORM / (norms + CLIP_EPS)).clamp(max=1.0)
    clipped = [(g.float().reshape(groups, -1) * scale[:, None]).to(g.dtype).view(g.shape) for g in grads]
    return {"grads": clipped, "norms": norms}


def _plain_norm(s, group, place):
    x, weight = s["x"].float(), s["weight"].float()
    centred = x - x.mean(dim=1, keepdim=True)
    scale = torch.rsqrt(centred.square().mean(dim=1, keepdim=True) + NORM_EPS)
    h = centred * scale
    if s["case"]["op"] == "norm_fwd":
        return (h * weight[group] + s["bias"].float()[group]).to(s["x"].dtype)
    g = s["grad_y"].float()
    q = g * weight[group]
    grad_x = scale * (q - q.mean(dim=1, keepdim=True) - h * (q * h).mean(dim=1, keepdim=True))
    return {
        "grad_x": grad_x.to(s["x"].dtype),
        "grad_weight": _padded(g * h, s, group, place).sum(dim=1).to(s["x"].dtype),
        "grad_bias": _padded(g, s, group, place).sum(dim=1).to(s["x"].dtype),
    }


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "clip":
        return _plain_clip(s)
    group, place = _slots(s)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _plain_norm(s, group, place)
    dtype, (groups, _, hidden, width) = s["x"].dtype, s["weight"].shape
    weight, bias = s["weight"].float().view(groups, 2 * hidden, width), s["bias"].float().view(groups, 2 * hidden)
    x = _padded(s["x"], s, group, place)
    both = torch.bmm(x, weight.transpose(1, 2).contiguous()) + bias[:, None]
    act, slope = _activated(both[:, :, :hidden], case["activation"])
    up = both[:, :, hidden:]
    if case["op"] == "gated_fwd":
        return (act * up)[group, place].to(dtype)
    g = _padded(s["grad_y"], s, group, place)
    back = torch.cat([g * up * slope, g * act], dim=2)
    return {
        "grad_x": torch.bmm(back, weight)[group, place].to(dtype),
        "grad_weight": torch.bmm(back.transpose(1, 2).contiguous(), x).view(groups, 2, hidden, width).to(dtype),
        "grad_bias": back.sum(dim=1).view(groups, 2, hidden).to(dtype),
    }


def work(case):
    if case["op"] == "clip":
        values = total = 0
        for s in _shapes(case):
            n = math.prod(s)
            size = {"float32": 4, "mixed": 2 if len(s) > 2 else 4}.get(case["dtype"], 2)
            values, total = values + n, total + n * size
        return {"bytes": 2 * total + 4 * (case["groups"] if case["per_group"] else 1), "flops": 3 * values}
    size = 4 if case["dtype"] == "float32" else 2
    rows, width, groups = case["rows"], case["width"], case["groups"]
    offsets, used = 8 * (groups + 1), min(groups, rows)
    if case["op"] == "norm_fwd":
        return {"bytes": size * (2 * rows * width + 2 * used * width) + offsets, "flops": 8 * rows * width}
    if case["op"] == "norm_bwd":
        return {"bytes": size * (3 * rows * width + used * width + 2 * groups * width) + offsets, "flops": 18 * rows * width}
    hidden = case["hidden"]
    if case["op"] == "gated_fwd":
        return {"bytes": size * (rows * (width + hidden) + 2 * used * hidden * (width + 1)) + offsets,
                "flops": 4 * rows * width * hidden}
    return {"bytes": size * (rows * (2 * width + hidden) + 2 * (used + groups) * hidden * (width + 1)) + offsets,
            "flops": 12 * rows * width * hidden}


def _exact_clip(s):
    case, grads = s["case"], s["grads"]
    groups = case["groups"] if case["per_group"] else 1
    norms = torch.zeros(groups, dtype=torch.float64, device="cuda")
    for g in grads:
        for n, part in enumerate(g.reshape(groups, -1)):
            norms[n] += torch.linalg.vector_norm(part.double()) ** 2
    norms = norms.sqrt()
    clipped = []
    for g in grads:
        flat = g.double().reshape(groups, -1)
        for n in range(groups):
            if MAX_NORM < norms[n] + CLIP_EPS:
                flat[n] *= MAX_NORM / (norms[n] + CLIP_EPS)
        clipped.append(flat.view(g.shape))
    return {"grads": clipped, "norms": norms}


def _exact_act(a, kind):
    """act(a) and act'(a) in 64 bits, the derivative from the definitions by the standard normal's density and the logistic's"""
    if kind == "gelu":
        below = 0.5 * torch.special.erfc(-a / math.sqrt(2.0))
        return a * below, below + a * torch.exp(-0.5 * a.square()) / math.sqrt(math.tau)
    if kind == "gelu_tanh":
        # 0.5 (1 + tanh z) = sigmoid(2 z)
        sig = torch.sigmoid(2.0 * GELU * a * (1.0 + 0.044715 * a.square()))
        return a * sig, sig + a * sig * (1.0 - sig) * 2.0 * GELU * (1.0 + 0.134145 * a.square())
    sig = torch.sigmoid(a)
    return (a * sig, sig + a * sig * (1.0 - sig)) if kind == "silu" else (sig, sig * (1.0 - sig))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        return _exact_clip(s)
    ends = s["row_offsets"].tolist()
    y, gx, gw, gb = [], [], [], []
    for n, (lo, hi) in enumerate(zip(ends, ends[1:])):
        x, w, b = s["x"][lo:hi].double(), s["weight"][n].double(), s["bias"][n].double()
        g = s["grad_y"][lo:hi].double() if "grad_y" in s else None
        if case["op"] in ("norm_fwd", "norm_bwd"):
            spread, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            deviation = torch.sqrt(spread + NORM_EPS)
            h = (x - mean) / deviation
            if g is None:
                y.append(h * w + b)
                continue
            q = g * w / deviation
            gx.append(q - q.mean(dim=1, keepdim=True) - h * (h * q).sum(dim=1, keepdim=True) / x.shape[1])
            gw.append((g * h).sum(dim=0))
            gb.append(g.sum(dim=0))
            continue
        (act, slope), up = _exact_act(x @ w[0].T + b[0], case["activation"]), x @ w[1].T + b[1]
        if g is None:
            y.append(act * up)
            continue
        da, du = g * slope * up, g * act
        gx.append(da @ w[0] + du @ w[1])
        gw.append(torch.stack([da.T @ x, du.T @ x]))
        gb.append(torch.stack([da.sum(dim=0), du.sum(dim=0)]))
    if "grad_y" not in s:
        return torch.cat(y)
    return {"grad_x": torch.cat(gx), "grad_weight": torch.stack(gw), "grad_bias": torch.stack(gb)}
