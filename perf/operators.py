"""The operators around the reduction, as a training step calls them, with the
sizes they are measured at.

A node's backward pass ends in layer norms whose weights' gradients go into the
node's row of the [P, N] gradients; the reduction's result goes into the
momentum; the momentum's matrices are orthogonalised and move the weights:

  layer_norm           y = (x - mean) * rstd * weight + bias over rows of D, also
                       after adding a residual stream, which is returned too
  layer_norm_backward  its gradients; the weight's and the bias's for each of P nodes
  momentum_step        m = mu * m + scale * g and the update (scale * g + mu * m with
                       Nesterov) from a reduction's result, sparse pairs or dense
  orthogonalize        every matrix of a flat update by Newton-Schulz products
  orthogonal_step      the same, then w = (1 - lr * decay) * w - lr * s * o in place,
                       s = sqrt(max(1, rows / cols))

`run` takes the plain form of each (torch operations in 32 bits) where `own` is
false, and this package's call where it is true. `exact` is the definition in
64 bits.
"""
import math

import torch

own = False

EPS = 1e-5                                   # of the layer norms
MU, SCALE = 0.95, 1.0 / 16                   # momentum, and the mean over 16 nodes
STEPS, COEFFICIENTS, NS_EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7
LR, DECAY = 0.02, 0.01

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of each of 8 sequences through a layer norm: latency
        {"name": "norm of 8 tokens", "op": "layer_norm", "rows": 8, "cols": 4096, "type": "bf16", "residual": False, "pad": 0},
        # ragged batch of an odd width, its rows a slice of a wider buffer
        {"name": "norm, odd, strided", "op": "layer_norm", "rows": 4099, "cols": 1537, "type": "f32", "residual": False, "pad": 63},
        # a training batch: the residual stream is added on the way
        {"name": "norm of 65536 tokens", "op": "layer_norm", "rows": 65536, "cols": 4096, "type": "bf16", "residual": True, "pad": 0},
        # the last few tokens of 4 nodes
        {"name": "gradients of 64 tokens", "op": "layer_norm_backward", "nodes": 4, "rows": 16, "cols": 1024, "type": "f32", "residual": False},
        # 3 nodes with an odd batch and a width that is no power of two
        {"name": "gradients, odd", "op": "layer_norm_backward", "nodes": 3, "rows": 1001, "cols": 1000, "type": "f16", "residual": False},
        # the training batch's backward pass, 8 nodes, the residual's gradient added on the way
        {"name": "gradients of 65536 tokens", "op": "layer_norm_backward", "nodes": 8, "rows": 8192, "cols": 4096, "type": "bf16", "residual": True},
        # the reduced gradient of the 272474-parameter network at 24% density: latency
        {"name": "momentum of 272474", "op": "momentum_step", "n": 272474, "density": 0.24, "dense": False, "type": "f32", "nesterov": True},
        # the wide network's reduced gradient: 64 nodes' 0.5% leave 27% of 2^27
        {"name": "momentum of 2^27", "op": "momentum_step", "n": 1 << 27, "density": 0.27, "dense": False, "type": "bf16", "nesterov": True},
        # every matrix of the 272474-parameter network, its weights moved in place: latency
        {"name": "step of 20 small layers", "op": "orthogonal_step", "shapes": "1x16x27,6x16x144,1x32x144,5x32x288,1x64x288,5x64x576,1x10x64", "from": "f32", "type": "f32"},
        # ragged matrices, wide and tall, whose sides no tile divides
        {"name": "orthogonalise, odd", "op": "orthogonalize", "shapes": "1x1000x1537,1x2049x513,2x257x771", "from": "f32", "type": "f32"},
        # the matrices of one transformer block of width 1024
        {"name": "orthogonalise a block", "op": "orthogonalize", "shapes": "4x1024x1024,1x4096x1024,1x1024x4096", "from": "f32", "type": "bf16"},
        # a large model's layers, weights in 16 bits
        {"name": "step of large layers", "op": "orthogonal_step", "shapes": "2x4096x4096,1x16384x4096", "from": "bf16", "type": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "momentum_step", "orthogonalize", "orthogonal_step"])
    kind = rng.choice(sorted(TYPES))
    if op == "layer_norm":
        cols = _log(rng, 16, 16384)
        rows = _log(rng, 1, max(2, (1 << 27) // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": kind, "residual": rng.random() < 0.5,
                "pad": rng.choice([0, 0, rng.randrange(1, 200)])}
    if op == "layer_norm_backward":
        cols = _log(rng, 16, 16384)
        rows = _log(rng, 4, max(5, (1 << 27) // cols))
        nodes = min(rows, rng.choice([1, 2, 3, 4, 8, 16, 64]))
        return {"op": op, "nodes": nodes, "rows": rows // nodes, "cols": cols, "type": kind, "residual": rng.random() < 0.5}
    if op == "momentum_step":
        return {"op": op, "n": _log(rng, 1 << 12, 1 << 27), "density": round(math.exp(rng.uniform(math.log(0.002), math.log(0.27))), 4),
                "dense": rng.random() < 0.3, "type": rng.choice(["bf16", "f32"]), "nesterov": rng.random() < 0.7}
    shapes, left = [], 4e12
    for _ in range(rng.randint(1, 3)):
        rows, cols, count = _log(rng, 16, 4096), _log(rng, 16, 8192), rng.randint(1, 6)
        count = min(count, int(left / _products(rows, cols)))
        if count:
            shapes.append("%dx%dx%d" % (count, rows, cols))
            left -= count * _products(rows, cols)
    return {"op": op, "shapes": ",".join(shapes), "from": rng.choice(["f32", "f32", "bf16"]), "type": kind}


# ---------------------------------------------------------------------------
def _groups(text):
    """[(first position, count, rows, cols)] of the matrices that follow each other in the flat update, and its length."""
    got, at = [], 0
    for part in text.split(","):
        count, rows, cols = (int(v) for v in part.split("x"))
        got.append((at, count, rows, cols))
        at += count * rows * cols
    return got, at


def _matrices(text):
    return [(at + k * rows * cols, rows, cols) for at, count, rows, cols in _groups(text)[0] for k in range(count)]


def _products(rows, cols):
    """Operations that the Newton-Schulz steps of one matrix cannot do without, with m <= n its sides. X moves only by
    polynomials of its Gram matrix, so the steps can be composed: half of the symmetric product X X^T, in each step the
    half of A A, for each further step three more symmetric products (the next A from this one, the polynomials'
    product), and all of B X once."""
    m, n = min(rows, cols), max(rows, cols)
    return 3 * m * m * n + (4 * STEPS - 3) * m * m * m


def _size(kind):
    return 4 if kind == "f32" else 2


def work(case):
    op = case["op"]
    if op == "layer_norm":
        e = case["rows"] * case["cols"]
        s = _size(case["type"])
        return {"bytes": e * s * (4 if case["residual"] else 2) + 8 * case["rows"] + 8 * case["cols"], "flops": 8 * e}
    if op == "layer_norm_backward":
        rows = case["nodes"] * case["rows"]
        e, s = rows * case["cols"], _size(case["type"])
        return {"bytes": e * s * (4 if case["residual"] else 3) + 8 * rows + 4 * case["cols"] + 8 * case["nodes"] * case["cols"],
                "flops": 14 * e}
    if op == "momentum_step":
        n = case["n"]
        g = 4 * n if case["dense"] else 8 * int(n * case["density"])
        return {"bytes": g + 8 * n + _size(case["type"]) * n, "flops": 5 * n}
    groups, n = _groups(case["shapes"])
    moved = _size(case["type"]) * (2 if op == "orthogonal_step" else 1)
    return {"bytes": n * (_size(case["from"]) + moved), "flops": sum(c * _products(r, k) for _, c, r, k in groups)}


# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    op, kind = case["op"], TYPES[case["type"]]
    s = {"case": case}
    if op == "layer_norm":
        rows, cols = case["rows"], case["cols"]
        x = (normal(rows, cols + case["pad"]) * 1.5 + 0.25).to(kind)
        s["x"] = x[:, :cols]
        s["residual"] = (normal(rows, cols) * 2 - 0.1).to(kind) if case["residual"] else None
        s["weight"], s["bias"] = 1 + 0.1 * normal(cols), 0.1 * normal(cols)
    elif op == "layer_norm_backward":
        nodes, rows, cols = case["nodes"], case["rows"], case["cols"]
        x = (normal(nodes, rows, cols) * 1.5 + 0.25).to(kind)
        s["x"], s["dy"] = x, normal(nodes, rows, cols).to(kind)
        s["dresidual"] = normal(nodes, rows, cols).to(kind) if case["residual"] else None
        s["weight"] = 1 + 0.1 * normal(cols)
        s["mean"] = x.float().mean(-1)
        s["rstd"] = torch.rsqrt((x.float() - s["mean"][..., None]).square().mean(-1) + EPS)
    elif op == "momentum_step":
        n = case["n"]
        s["momentum"] = normal(n) * 1e-3
        keep = torch.rand(n, generator=gen, device=dev) < case["density"]
        idx = keep.nonzero().view(-1).to(torch.int32)
        s["count"] = idx.numel()
        value = normal(n) * 2e-3  # what the Top-k sends is never near zero
        value += torch.copysign(torch.full_like(value, 4e-3), value)
        s["value"] = torch.where(keep, value, torch.zeros_like(value))
        s["index"] = torch.full((max(1, int(0.35 * n)),), -1, dtype=torch.int32, device=dev)
        if not case["dense"]:  # the pairs, then what the reduction leaves unwritten
            s["index"][: s["count"]] = idx
            s["value"][: s["count"]] = value[keep]
        # the reduction's record: pairs in the union, whether the result is dense, input flags
        s["result"] = torch.tensor([s["count"], int(case["dense"])], dtype=torch.int64, device=dev).view(torch.uint8)
    else:
        groups, n = _groups(case["shapes"])
        update = torch.empty(n, device=dev)
        for at, count, rows, cols in groups:  # noise, and a few directions that stand out of it
            g = normal(count, rows, cols)
            for i in range(3):
                g += (4.0 / (i + 1)) * normal(count, rows, 1) * normal(count, 1, cols)
            update[at: at + count * rows * cols] = 1e-3 * g.view(-1)
        s["update"] = update.to(TYPES[case["from"]])
        if op == "orthogonal_step":
            s["weight"] = (normal(n) * 0.02).to(kind)
    return s


# ---------------------------------------------------------------------------
def _layer_norm(s):
    x, t = s["x"], s["x"].dtype
    a = x.float()
    if s["residual"] is not None:
        total = (a + s["residual"].float()).to(t)
        a = total.float()
    mean = a.mean(-1)
    c = a - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(-1) + EPS)
    out = {"y": (c * rstd[:, None] * s["weight"] + s["bias"]).to(t), "mean": mean, "rstd": rstd}
    if s["residual"] is not None:
        out["total"] = total
    return out


def _layer_norm_backward(s):
    dy = s["dy"].float()
    h = (s["x"].float() - s["mean"][..., None]) * s["rstd"][..., None]
    d = dy * s["weight"]
    dx = s["rstd"][..., None] * (d - d.mean(-1, keepdim=True) - h * (d * h).mean(-1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(1), "dbias": dy.sum(1)}


def _momentum_step(s):
    case, m = s["case"], s["momentum"]
    m.mul_(MU)
    if case["dense"]:
        m.add_(s["value"], alpha=SCALE)
        u = m * MU + SCALE * s["value"] if case["nesterov"] else m
    else:
        k = s["count"]
        idx, g = s["index"][:k], s["value"][:k] * SCALE
        m.index_add_(0, idx, g)
        u = (m * MU).index_add_(0, idx, g) if case["nesterov"] else m
    return {"momentum": m, "update": u.to(TYPES[case["type"]]) if case["type"] != "f32" or case["nesterov"] else u.clone()}


def _newton_schulz(g):
    """[count, rows, cols] -> nearly orthogonal matrices of the same shape."""
    a, b, c = COEFFICIENTS
    tall = g.shape[1] > g.shape[2]
    x = g.float()
    if tall:
        x = x.transpose(1, 2).contiguous()
    norm = torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True, dtype=torch.float64)
    x = x / (norm.float() + NS_EPS)
    for _ in range(STEPS):
        p = torch.bmm(x, x.transpose(1, 2).contiguous())
        q = torch.baddbmm(p, p, p, beta=b, alpha=c)
        x = torch.baddbmm(x, q, x, beta=a)
    return x.transpose(1, 2) if tall else x


def _orthogonal(s):
    case = s["case"]
    kind, step = TYPES[case["type"]], case["op"] == "orthogonal_step"
    out = s["weight"] if step else torch.empty(s["update"].shape, dtype=kind, device=s["update"].device)
    for at, count, rows, cols in _groups(case["shapes"])[0]:
        there = slice(at, at + count * rows * cols)
        o = _newton_schulz(s["update"][there].view(count, rows, cols)).reshape(-1)
        if step:
            o = (1 - LR * DECAY) * out[there].float() - LR * math.sqrt(max(1.0, rows / cols)) * o
        out[there] = o.to(kind)
    return {"weight" if step else "out": out}


def _own(s):
    import sparse_gradient_reduction_amd as sg

    case = s["case"]
    op = case["op"]
    if op == "layer_norm":
        if s["residual"] is None:
            y, mean, rstd = sg.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        y, mean, rstd, total = sg.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"])
        return {"y": y, "mean": mean, "rstd": rstd, "total": total}
    if op == "layer_norm_backward":
        dx, dweight, dbias = sg.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                                    nodes=case["nodes"], dresidual=s["dresidual"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "momentum_step":
        reduced = sg.ReduceOutput(s["result"], s["index"], s["value"], case["n"])
        u = sg.momentum_step(reduced, s["momentum"], MU, scale=SCALE, nesterov=case["nesterov"], dtype=TYPES[case["type"]])
        return {"momentum": s["momentum"], "update": u}
    matrices = _matrices(case["shapes"])
    if op == "orthogonal_step":
        sg.orthogonal_step(s["weight"], s["update"], matrices, lr=LR, weight_decay=DECAY, steps=STEPS,
                           coefficients=COEFFICIENTS, eps=NS_EPS)
        return {"weight": s["weight"]}
    return {"out": sg.orthogonalize(s["update"], matrices, dtype=TYPES[case["type"]], steps=STEPS,
                                    coefficients=COEFFICIENTS, eps=NS_EPS)}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "layer_norm":
        return _layer_norm(state)
    if op == "layer_norm_backward":
        return _layer_norm_backward(state)
    if op == "momentum_step":
        return _momentum_step(state)
    return _orthogonal(state)


# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "layer_norm":
        v = s["x"].double()
        out = {}
        if s["residual"] is not None:
            v = v + s["residual"].double()
            out["total"] = v
            v = v.to(s["x"].dtype).double()  # the norm is that of the sum as it is stored
        var, mean = torch.var_mean(v, dim=1, correction=0)
        out["mean"], out["rstd"] = mean, 1 / torch.sqrt(var + EPS)
        out["y"] = torch.addcmul(s["bias"].double(), (v - mean[:, None]) / torch.sqrt(var + EPS)[:, None], s["weight"].double())
        return out
    if op == "layer_norm_backward":
        # along x: y_i = w_i * (x_i - mean) * rstd, so dL/dx = rstd * P(w * dy), P the projection off 1 and off xhat
        r = s["rstd"].double().unsqueeze(2)
        xhat = (s["x"].double() - s["mean"].double().unsqueeze(2)) * r
        dy = s["dy"].double()
        wdy = dy * s["weight"].double()
        one = wdy.sum(2, keepdim=True) / case["cols"]
        hat = (wdy * xhat).sum(2, keepdim=True) / case["cols"]
        dx = (wdy - one - xhat * hat) * r
        if s["dresidual"] is not None:
            dx += s["dresidual"].double()
        return {"dx": dx, "dweight": (dy * xhat).sum(1), "dbias": dy.sum(1)}
    if op == "momentum_step":
        g = s["value"].double()
        if not case["dense"]:
            g = torch.zeros_like(g)
            g[s["index"][: s["count"]].long()] = s["value"][: s["count"]].double()
        g = g * SCALE
        m = MU * s["momentum"].double() + g
        return {"momentum": m, "update": g + MU * m if case["nesterov"] else m}
    a, b, c = COEFFICIENTS
    step = op == "orthogonal_step"
    out = s["weight"].double() if step else torch.empty(s["update"].shape, dtype=torch.float64, device=s["update"].device)
    for at, rows, cols in _matrices(case["shapes"]):
        x = s["update"][at: at + rows * cols].view(rows, cols).double()
        x = x / (torch.sqrt((x * x).sum()) + NS_EPS)
        for _ in range(STEPS):
            if rows <= cols:
                k = x @ x.t()
                x = a * x + (b * k + c * (k @ k)) @ x
            else:
                k = x.t() @ x
                x = a * x + x @ (b * k + c * (k @ k))
        there = out[at: at + rows * cols]
        if step:
            there.mul_(1 - LR * DECAY).sub_(x.reshape(-1), alpha=LR * math.sqrt(max(1.0, rows / cols)))
        else:
            there.copy_(x.reshape(-1))
    return {"weight" if step else "out": out}
