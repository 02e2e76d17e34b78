"""The per-mesh layers and their optimiser step: what they compute, and on what sizes they are measured.

Two operators, on packed batches in the layout of the rest of the library (rows of all groups one after another, and
row_offsets [N + 1]: group n owns rows [row_offsets[n], row_offsets[n + 1])):

  grouped_linear  y_r = W_n x_r + b_n for every row r of group n, with one weight [out, in] and one bias [out] per group,
                  and its backward pass: grad_x_r = W_n^T g_r, grad_W_n = sum_r g_r x_r^T, grad_b_n = sum_r g_r.
  orthogonalize   X_0 = U / (|U|_F + eps); X <- a X + (b A + c A A) X with A = X X^T, (a, b, c) = (3.4445, -4.7750,
                  2.0315), `steps` times, for every matrix U of a batch [B, m, n].

`run` computes them in their plain form (elementary torch operations in 32 bits) where `own` is false, and through the
library's entry points where it is true.
"""

import math
import random

import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
STEPS = 5


def listed():
    return [
        # A decoder's hidden layer on one token per mesh: the smallest call, all latency.
        dict(name="fwd 8x1 rows 64-64 f16", op="fwd", dtype="float16", groups=8, layout="one", rows=8, cin=64, cout=64),
        # One query row for each of 64 groups against wide weights, as an autoregressive head calls it: weights are streamed.
        dict(name="fwd 64x1 rows 1024 bf16", op="fwd", dtype="bfloat16", groups=64, layout="one", rows=64, cin=1024, cout=1024),
        # The head that turns 64 features of each vertex into its offset, on the 16-sphere batch's vertex counts.
        dict(name="fwd spheres 64-3 f32", op="fwd", dtype="float32", groups=16, layout="levels", rows=217632, cin=64, cout=3),
        # Shading every pixel of 16 images of 256 x 256 with its own mesh's layer.
        dict(name="fwd pixels 64-64 bf16", op="fwd", dtype="bfloat16", groups=16, layout="even", rows=1 << 20, cin=64, cout=64),
        # Wide layers over ragged groups: the largest call.
        dict(name="fwd ragged 2048 bf16", op="fwd", dtype="bfloat16", groups=32, layout="ragged", rows=131072, cin=2048, cout=2048),
        # Odd widths, a few short groups and empty ones: nothing is aligned.
        dict(name="bwd odd 37-19 f16", op="bwd", dtype="float16", groups=7, layout="ragged", rows=1003, cin=37, cout=19),
        # Training the hidden layer of the vertex decoder on the 16-sphere batch, in the rasterizer's own type.
        dict(name="bwd spheres 64-64 f32", op="bwd", dtype="float32", groups=16, layout="levels", rows=217632, cin=64, cout=64),
        # Training wide layers over ragged groups.
        dict(name="bwd ragged 1024 bf16", op="bwd", dtype="bfloat16", groups=32, layout="ragged", rows=65536, cin=1024, cout=1024),
        # The update of the vertex heads of 16 meshes: the smallest matrices.
        dict(name="orth 16x3x64 f32", op="orth", dtype="float32", batch=16, m=3, n=64),
        # The update of an ordinary hidden layer of 16 decoders.
        dict(name="orth 16x256x256 f32", op="orth", dtype="float32", batch=16, m=256, n=256),
        # The update of eight wide layers kept in 16 bits.
        dict(name="orth 8x1024x1024 bf16", op="orth", dtype="bfloat16", batch=8, m=1024, n=1024),
        # The widest update, in 32 bits.
        dict(name="orth 4x2048x2048 f32", op="orth", dtype="float32", batch=4, m=2048, n=2048),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    if rng.random() < 0.35:
        m, n = _log_uniform(rng, 1, 2048), _log_uniform(rng, 1, 2048)
        if rng.random() < 0.3:
            m, n = (m + 63) // 64 * 64, (n + 63) // 64 * 64
        short, long_ = min(m, n), max(m, n)
        batch = _log_uniform(rng, 1, 32)
        while batch > 1 and batch * short * short * (3 * long_ + short) > 4 * 4 * 2048**3:
            batch //= 2
        return dict(op="orth", dtype=rng.choice(list(DTYPES)), batch=batch, m=m, n=n)
    op = rng.choice(["fwd", "bwd"])
    cin, cout = _log_uniform(rng, 3, 2048), _log_uniform(rng, 3, 2048)
    if rng.random() < 0.5:
        cin, cout = (cin + 15) // 16 * 16, (cout + 15) // 16 * 16
    groups = _log_uniform(rng, 1, 128)
    layout = rng.choice(["one", "even", "ragged", "ragged", "levels"])
    dtype = rng.choice(list(DTYPES))
    if layout == "one":
        return dict(op=op, dtype=dtype, groups=groups, layout=layout, rows=groups, cin=cin, cout=cout)
    passes = 1 if op == "fwd" else 2
    most = min(1 << 20, (1 << 39) // (cin * cout * passes), (1 << 27) // ((cin + cout) * passes))
    if layout == "levels":
        groups = rng.randint(1, 16)
        while groups > 1 and _levels_total(groups) > most:
            groups -= 1
        return dict(op=op, dtype=dtype, groups=groups, layout=layout, rows=_levels_total(groups), cin=cin, cout=cout)
    rows = _log_uniform(rng, 1, max(1, most))
    if layout == "even":
        rows = max(1, rows // groups) * groups
    return dict(op=op, dtype=dtype, groups=groups, layout=layout, rows=rows, cin=cin, cout=cout)


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    state = dict(case=case)
    if case["op"] == "orth":
        # momentum of a layer's gradients: a few strong directions over noise, small in scale
        batch, m, n = case["batch"], case["m"], case["n"]
        rank = max(1, min(m, n) // 8)
        strong = torch.bmm(_normal((batch, m, rank), gen), _normal((batch, rank, n), gen)) / math.sqrt(rank)
        state["update"] = ((strong + 0.1 * _normal((batch, m, n), gen)) * 1e-2).to(dtype)
        return state
    sizes = _group_sizes(case, seed)
    groups, rows, cin, cout = case["groups"], case["rows"], case["cin"], case["cout"]
    offsets = [0]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    state["longest"] = max(sizes)
    state["row_offsets"] = torch.tensor(offsets, dtype=torch.int64, device="cuda")
    state["x"] = _normal((rows, cin), gen).clamp_(min=0.0).to(dtype)  # features after a rectifier
    state["weight"] = (_normal((groups, cout, cin), gen) / math.sqrt(cin)).to(dtype)
    state["bias"] = (0.1 * _normal((groups, cout), gen)).to(dtype)
    if case["op"] == "bwd":
        covered = torch.rand((rows, 1), generator=gen, device="cuda") < 0.7  # rows that no pixel sees get no gradient
        state["grad_y"] = (_normal((rows, cout), gen) * covered).to(dtype)
    return state


def _run_own(s):
    import differentiable_mesh_rasterization_amd as dmr

    if s["case"]["op"] == "orth":
        return dmr.orthogonalize(s["update"], steps=STEPS, eps=EPS)
    x, row_offsets, weight = s["x"], s["row_offsets"], s["weight"]
    if s["case"]["op"] == "fwd":
        return dmr.grouped_linear(x, row_offsets, weight, s["bias"])
    groups, cout, cin = weight.shape
    grads = {"grad_x": torch.empty_like(x), "grad_weight": torch.empty_like(weight), "grad_bias": torch.empty_like(s["bias"])}
    size = dmr.dmr_grouped_linear_workspace_size(x.shape[0], groups, cin, cout, x.dtype)
    workspace = torch.empty(size, dtype=torch.uint8, device=x.device)
    dmr.dmr_grouped_linear_bwd(x, row_offsets, weight, s["grad_y"], workspace=workspace, **grads)
    return grads


def _plain_step(x):
    a, b, c = COEFFICIENTS
    gram = torch.bmm(x, x.transpose(1, 2))
    poly = b * gram + c * torch.bmm(gram, gram)
    return a * x + torch.bmm(poly, x)


def _plain_orthogonalize(update):
    x = update.float()
    if x.shape[1] > x.shape[2]:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    x = _plain_step(_plain_step(_plain_step(_plain_step(_plain_step(x)))))
    return (x.transpose(1, 2) if update.shape[1] > update.shape[2] else x).to(update.dtype).contiguous()


def _slots(s):
    """Each row's group and its place within it, for products over groups padded to the longest."""
    offsets = s["row_offsets"]
    row = torch.arange(s["x"].shape[0], device="cuda")
    group = torch.searchsorted(offsets[1:], row, right=True)
    return group, row - offsets[group]


def _padded(v, s, group, place):
    wide = torch.zeros((s["weight"].shape[0], s["longest"], v.shape[1]), dtype=torch.float32, device="cuda")
    wide[group, place] = v.float()
    return wide


def run(s):
    if own:
        return _run_own(s)
    if s["case"]["op"] == "orth":
        return _plain_orthogonalize(s["update"])
    group, place = _slots(s)
    weight = s["weight"].float()
    x = _padded(s["x"], s, group, place)
    if s["case"]["op"] == "fwd":
        y = torch.bmm(x, weight.transpose(1, 2))[group, place]
        return (y + s["bias"].float()[group]).to(s["x"].dtype)
    g = _padded(s["grad_y"], s, group, place)
    return {
        "grad_x": torch.bmm(g, weight)[group, place].to(s["x"].dtype),
        "grad_weight": torch.bmm(g.transpose(1, 2), x).to(s["x"].dtype),
        "grad_bias": g.sum(dim=1).to(s["x"].dtype),
    }


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "orth":
        # X X^T and A A are symmetric: half of their products are enough
        batch, short, long_ = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
        step = short * (short + 1) * long_ + short * (short + 1) * short + 2 * short * short * long_
        return {"bytes": 2 * batch * short * long_ * size, "flops": batch * STEPS * step}
    rows, cin, cout, groups = case["rows"], case["cin"], case["cout"], case["groups"]
    weights = groups * cout * cin
    if case["layout"] == "ragged":
        weights = min(groups, rows) * cout * cin
    vectors = groups * cout
    offsets = 8 * (groups + 1)
    if case["op"] == "fwd":
        return {"bytes": size * (rows * (cin + cout) + weights + vectors) + offsets, "flops": 2 * rows * cin * cout}
    return {"bytes": size * (rows * (2 * cin + cout) + weights + groups * cout * cin + vectors) + offsets,
            "flops": 4 * rows * cin * cout + rows * cout}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orth":
        a, b, c = COEFFICIENTS
        results = []
        for u in s["update"].double():
            u = u / (torch.linalg.matrix_norm(u) + EPS)
            wide = u.shape[0] <= u.shape[1]
            for _ in range(STEPS):
                gram = u @ u.T if wide else u.T @ u
                second = gram @ u if wide else u @ gram
                fourth = gram @ second if wide else second @ gram
                u = a * u + b * second + c * fourth
            results.append(u)
        return torch.stack(results)
    ends = s["row_offsets"].tolist()
    y, gx, gw, gb = [], [], [], []
    for n, (lo, hi) in enumerate(zip(ends, ends[1:])):
        x, w = s["x"][lo:hi].double(), s["weight"][n].double()
        if case["op"] == "fwd":
            y.append(x @ w.T + s["bias"][n].double())
        else:
            g = s["grad_y"][lo:hi].double()
            gx.append(g @ w)
            gw.append(g.T @ x)
            gb.append(g.sum(dim=0))
    if case["op"] == "fwd":
        return torch.cat(y)
    return {"grad_x": torch.cat(gx), "grad_weight": torch.stack(gw), "grad_bias": torch.stack(gb)}
