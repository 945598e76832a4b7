"""The operators of a self-attention's training step, as a data-parallel program
calls them between its products, with the sizes they are measured at.

A block projects its normed rows to queries, keys and values, norms the queries
and keys of every head and rotates them by their positions, attends, and in the
backward pass takes the gradients the same way back; the norms' weights get one
gradient for each of P nodes, like layer norm's:

  head_norm_rotate           q, k over their heads' D elements: x / sqrt(mean x^2 + eps) * weight,
                             then pairs of elements turned by position * frequency
  head_norm_rotate_backward  its gradients; the weights' for each of P nodes
  attention                  softmax(scale * q k^T over what a query sees) v, and the
                             logarithm of each row's sum of exponentials
  attention_backward         the gradients of q, k and v from those, the
                             probabilities computed again

A query at place i of a sequence of n queries and m keys sees the keys j with
i + m - n - window < j (< i + m - n + window, or <= i + m - n where causal).

`run` takes the plain form of each (torch operations in 32 bits, angles in 64)
where `own` is false, and this package's call where it is true. `exact` is the
definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0          # of the rotation's frequencies BASE^(-2 i / rotated)

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _attention(op, name, batch, queries, keys, heads, groups, dim, kind, causal, window=0, lengths=""):
    return {"name": name, "op": op, "batch": batch, "queries": queries, "keys": keys, "heads": heads, "groups": groups,
            "dim": dim, "type": kind, "causal": causal, "window": window, "lengths": lengths}


def _norms(op, name, nodes, rows, heads, groups, dim, rotated, kind, first=0, interleaved=False):
    return {"name": name, "op": op, "nodes": nodes, "rows": rows, "heads": heads, "groups": groups, "dim": dim,
            "rotated": rotated, "type": kind, "first": first, "interleaved": interleaved}


def listed():
    a, b = "attention", "attention_backward"
    n, g = "head_norm_rotate", "head_norm_rotate_backward"
    ragged = "1001,640,0,17,999"
    return [
        # short sequences of a block of width 1024: latency
        _attention(a, "attention of 8 x 64 tokens", 8, 64, 64, 16, 16, 64, "bf16", True),
        # a padded batch with an empty sequence, a sliding window, shared heads whose width no tile divides
        _attention(a, "attention, odd, padded", 5, 1001, 1001, 12, 4, 80, "f16", True, 300, ragged),
        # a few learned queries that read a long sequence
        _attention(a, "attention of 65 queries", 2, 65, 16384, 8, 8, 64, "bf16", False),
        # a training batch of width 4096 with shared key and value heads
        _attention(a, "attention of 16384 tokens", 4, 4096, 4096, 32, 8, 128, "bf16", True),
        # the same four kinds backwards: short sequences
        _attention(b, "gradients of 8 x 64 tokens", 8, 64, 64, 16, 16, 64, "bf16", True),
        # the padded batch
        _attention(b, "gradients, odd, padded", 5, 1001, 1001, 12, 4, 80, "f16", True, 300, ragged),
        # one sequence's queries over another's keys, padded, in full precision
        _attention(b, "gradients across, fp32", 3, 333, 1500, 8, 8, 64, "f32", False, 0, "1500,700,1"),
        # the training batch
        _attention(b, "gradients of 16384 tokens", 4, 4096, 4096, 32, 8, 128, "bf16", True),
        # one token of each of 8 sequences, far into them: latency
        _norms(n, "head norms of 8 tokens", 1, 8, 16, 16, 64, 64, "bf16", 100000),
        # a training batch's queries and keys, slices of one projection
        _norms(n, "head norms of 65536 tokens", 1, 65536, 32, 8, 128, 128, "bf16"),
        # 3 nodes with an odd batch, half of every head rotated
        _norms(g, "their gradients, odd", 3, 1001, 6, 2, 80, 40, "f32", 7, True),
        # the training batch's, 8 nodes
        _norms(g, "their gradients, 65536 tokens", 8, 8192, 32, 8, 128, 128, "bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_backward", "attention_backward", "head_norm_rotate",
                     "head_norm_rotate_backward"])
    kind = rng.choice(["bf16", "bf16", "bf16", "f16", "f16", "f32"])
    dim = rng.choice([32, 40, 64, 64, 80, 96, 128, 128, rng.randrange(8, 129)])
    groups = _log(rng, 1, 16)
    heads = groups * rng.choice([1, 1, 2, 3, 4, 8])
    if op.startswith("head_norm"):
        nodes = 1 if op == "head_norm_rotate" else rng.choice([1, 2, 3, 4, 8, 16, 64])
        rows = _log(rng, 1, max(2, (1 << 28) // (dim * (heads + groups) * nodes)))
        return {"op": op, "nodes": nodes, "rows": rows, "heads": heads, "groups": groups, "dim": dim,
                "rotated": rng.choice([dim // 2 * 2, dim // 2 * 2, dim // 4 * 2, 0]), "type": kind,
                "first": rng.choice([0, 0, _log(rng, 1, 10000000)]), "interleaved": rng.random() < 0.4}
    # sequences from one token on; those of a training batch, whose gradients are wanted, from 16 on
    least = 16 if op == "attention_backward" else 1
    keys = _log(rng, least, 16384)
    queries = keys if rng.random() < 0.6 else _log(rng, 1, 16384)
    most = (1 << 31) // (32 if kind == "f32" else 4)   # pairs of a query and a key over all heads
    while queries * keys * heads > most:
        queries, keys = (queries + 1) // 2, keys if keys < 2 * least else (keys + 1) // 2
        if rng.random() < 0.5 and heads > groups:
            heads -= groups
    batch = max(1, min(_log(rng, 1, 64), most // (queries * keys * heads)))
    lengths = ""
    if rng.random() < 0.4:
        lengths = ",".join(str(rng.choice([keys, rng.randrange(keys + 1), rng.randrange(keys // 2, keys + 1)]) if x else keys)
                           for x in range(batch))
    return {"op": op, "batch": batch, "queries": queries, "keys": keys, "heads": heads, "groups": groups, "dim": dim,
            "type": kind, "causal": queries <= keys and rng.random() < 0.7,
            "window": _log(rng, least, 4096) if rng.random() < 0.3 else 0, "lengths": lengths}


# ---------------------------------------------------------------------------
def _size(kind):
    return 4 if kind == "f32" else 2


def _itself(case):
    """Whether the sequences attend to themselves: their queries are padded like their keys."""
    return case["queries"] == case["keys"]


def _lengths(case):
    """[(queries, keys)] of the sequences."""
    n, m = case["queries"], case["keys"]
    if not case["lengths"]:
        return [(n, m)] * case["batch"]
    return [(k if _itself(case) else n, k) for k in (int(v) for v in case["lengths"].split(","))]


def _seen(n, m, causal, window):
    """Pairs of a query and a key that it sees."""
    total, off, w = 0, m - n, window or 1 << 40
    for i in range(n):
        last = min(m - 1, i + off + (0 if causal else w - 1))
        total += max(0, last - max(0, i + off - w + 1) + 1)
    return total


def work(case):
    op, s, d, h, g = case["op"], _size(case["type"]), case["dim"], case["heads"], case["groups"]
    if op.startswith("head_norm"):
        rows, back = case["nodes"] * case["rows"], op.endswith("backward")
        e = rows * (h + g) * d
        return {"bytes": e * s * (3 if back else 2) + 4 * rows + 8 * d + (8 * d * case["nodes"] if back else 0) + 4 * case["rotated"],
                "flops": e * (14 if back else 7)}
    back = op.endswith("backward")
    lengths = _lengths(case)
    n, m = sum(v for v, _ in lengths), sum(v for _, v in lengths)
    all_n, all_m = case["batch"] * case["queries"], case["batch"] * case["keys"]
    pairs = sum(_seen(a, b, case["causal"], case["window"]) for a, b in lengths) * h
    if back:  # reads q, out, dout, lse, k, v; writes dq, dk, dv
        return {"bytes": s * d * (3 * n * h + all_n * h + 2 * (m + all_m) * g) + 4 * n * h, "flops": 10 * d * pairs}
    return {"bytes": s * d * (n * h + all_n * h + 2 * m * g) + 4 * all_n * h, "flops": 4 * d * pairs}


# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind = TYPES[case["type"]]
    h, g, d = case["heads"], case["groups"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = {"case": case}
    if case["op"].startswith("head_norm"):
        rows = case["nodes"] * case["rows"]
        # queries, keys and values of one projection
        every = (normal(rows, h + 2 * g, d) * (0.5 + torch.rand((rows, 1, 1), generator=gen, device=dev))).to(kind)
        s["q"], s["k"] = every[:, :h], every[:, h: h + g]
        s["qw"], s["kw"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
        s["position"] = (case["first"] + torch.arange(rows, device=dev) % 4096).to(torch.int32)
        r = case["rotated"]
        s["frequency"] = BASE ** (-2.0 * torch.arange(r // 2, device=dev, dtype=torch.float64) / max(r, 1)) if r else None
        if case["op"].endswith("backward"):
            s["dq"], s["dk"] = normal(rows, h, d).to(kind), normal(rows, g, d).to(kind)
        return s
    b, n, m = case["batch"], case["queries"], case["keys"]
    if _itself(case):  # of one projection
        every = normal(b, n, h + 2 * g, d)
        every[:, :, :h] *= 1.5
        s["q"], s["k"], s["v"] = every.to(kind).split((h, g, g), 2)
    else:
        s["q"], s["k"], s["v"] = (1.5 * normal(b, n, h, d)).to(kind), normal(b, m, g, d).to(kind), normal(b, m, g, d).to(kind)
    s["scale"] = d ** -0.5
    s["n"] = s["m"] = None
    if case["lengths"]:
        n, m = (torch.tensor(v, dtype=torch.int32, device=dev) for v in zip(*_lengths(case)))
        s["n"], s["m"] = (n if _itself(case) else None), m
    if case["op"] == "attention_backward":
        s["dout"] = normal(*s["q"].shape).to(kind)
        s["out"], s["lse"] = _forward(s)
    return s


# ---------------------------------------------------------------------------
def _turned(x, s, back):
    """The rotation of fp32 [rows, heads, D], or the one back."""
    r = 0 if s["frequency"] is None else 2 * s["frequency"].numel()
    if r == 0:
        return x
    angle = s["position"].double()[:, None] * s["frequency"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if back:
        sin = -sin
    if s["case"]["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        both = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        both = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return both if r == x.shape[-1] else torch.cat((both, x[..., r:]), -1)


def _head_norm_rotate(s):
    out = {}
    for name, weight in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
        out[name] = _turned(x, s, False).to(s[name].dtype)
    return out


def _head_norm_rotate_backward(s):
    out = {}
    for name, dy, weight in (("q", s["dq"], s["qw"]), ("k", s["dk"], s["kw"])):
        x, u = s[name].float(), _turned(dy.float(), s, True)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        x = x * r
        out["dweight " + name] = (u * x).view(s["case"]["nodes"], -1, x.shape[-1]).sum(1)
        u = u * weight
        out["d" + name] = (r * (u - x * (u * x).mean(-1, keepdim=True))).to(dy.dtype)
    return out


def _hidden(s):
    """[batch or 1, 1, queries, keys], true where a query does not see a key."""
    case, dev = s["case"], s["q"].device
    i = torch.arange(case["queries"], device=dev)[:, None]
    j = torch.arange(case["keys"], device=dev)
    n = torch.tensor([case["queries"]], device=dev) if s["n"] is None else s["n"]
    m = torch.tensor([case["keys"]], device=dev) if s["m"] is None else s["m"]
    n, m = n.view(-1, 1, 1, 1), m.view(-1, 1, 1, 1)
    place = i + m - n
    hide = (i >= n) | (j >= m)
    if case["causal"]:
        hide = hide | (j > place)
    if case["window"]:
        hide = hide | (j <= place - case["window"])
        if not case["causal"]:
            hide = hide | (j >= place + case["window"])
    return hide


def _by_heads(x, heads):
    """fp32 [batch, heads, rows, D] of [batch, rows, groups, D]."""
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(heads // x.shape[1], 1).contiguous()


def _forward(s):
    h = s["case"]["heads"]
    q, k, v = (_by_heads(s[x], h) for x in "qkv")
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    score.masked_fill_(_hidden(s), -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, v) / torch.where(total == 0, 1.0, total)
    return out.transpose(1, 2).to(s["q"].dtype).contiguous(), (top + torch.log(total))[..., 0]


def _backward(s):
    case, t = s["case"], s["q"].dtype
    h, g = case["heads"], case["groups"]
    q, k, v, do, o = (_by_heads(s[x], h) for x in ("q", "k", "v", "dout", "out"))
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    p.masked_fill_(_hidden(s), -math.inf)
    p.sub_(torch.where(s["lse"] == -math.inf, 0.0, s["lse"])[..., None]).exp_()

    def rows(x):  # [batch, heads, rows, D] -> [batch, rows, groups, D], a group's heads added up
        return x.view(x.shape[0], g, -1, *x.shape[2:]).sum(2).transpose(1, 2).to(t).contiguous()

    dv = rows(torch.matmul(p.transpose(2, 3).contiguous(), do))
    ds = torch.matmul(do, v.transpose(2, 3).contiguous()).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k).transpose(1, 2).to(t).contiguous()
    return {"dq": dq, "dk": rows(torch.matmul(ds.transpose(2, 3).contiguous(), q)), "dv": dv}


def _own(s):
    import sparse_gradient_reduction_amd as sg

    case = s["case"]
    op = case["op"]
    if op == "head_norm_rotate":
        q, k = sg.head_norm_rotate(s["q"], s["k"], s["qw"], s["kw"], s["position"], s["frequency"], eps=EPS,
                                   interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "head_norm_rotate_backward":
        dq, dk, dqw, dkw = sg.head_norm_rotate_backward(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["position"],
                                                        s["frequency"], eps=EPS, interleaved=case["interleaved"],
                                                        nodes=case["nodes"])
        return {"dweight q": dqw, "dq": dq, "dweight k": dkw, "dk": dk}
    mask = {"causal": case["causal"], "window": case["window"] or None, "scale": s["scale"], "q_lengths": s["n"],
            "k_lengths": s["m"]}
    if op == "attention":
        out, lse = sg.attention(s["q"], s["k"], s["v"], **mask)
        return {"out": out, "lse": lse}
    dq, dk, dv = sg.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], **mask)
    return {"dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "head_norm_rotate":
        return _head_norm_rotate(state)
    if op == "head_norm_rotate_backward":
        return _head_norm_rotate_backward(state)
    if op == "attention":
        out, lse = _forward(state)
        return {"out": out, "lse": lse}
    return _backward(state)


# ---------------------------------------------------------------------------
def _exact_norms(s):
    """Pairs of elements as complex numbers, turned by multiplication with e^(i angle)."""
    case = s["case"]
    r, back = case["rotated"], case["op"].endswith("backward")

    def pairs(x):
        c = x[..., :r].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
        return torch.complex(c[..., 0], c[..., 1])

    def turn(x, sign):
        if r == 0:
            return x
        angle = sign * torch.outer(s["position"].double(), s["frequency"])
        c = torch.view_as_real(pairs(x) * torch.polar(torch.ones_like(angle), angle)[:, None])
        c = c if case["interleaved"] else c.transpose(-1, -2)
        return torch.cat((c.flatten(-2), x[..., r:]), -1)

    out = {}
    for name, weight in (("q", s["qw"].double()), ("k", s["kw"].double())):
        x = s[name].double()
        size = torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
        if not back:
            out[name] = turn(x * weight / size, 1)
            continue
        u = turn(s["d" + name].double(), -1)
        out["dweight " + name] = (u * x / size).unflatten(0, (case["nodes"], -1)).sum((1, 2))
        # d(x / size): the part along x shrinks by what the size takes
        wu = weight * u
        out["d" + name] = wu / size - x * ((wu * x).sum(-1, keepdim=True) / case["dim"]) / size ** 3
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("head_norm"):
        return _exact_norms(s)
    back = case["op"] == "attention_backward"
    b, n, h, d = s["q"].shape
    m, g = case["keys"], case["groups"]
    dev, f64 = s["q"].device, torch.float64
    out, lse = torch.zeros((b, n, h, d), dtype=f64, device=dev), torch.full((b, h, n), -math.inf, dtype=f64, device=dev)
    dq, dk, dv = torch.zeros_like(out), torch.zeros((b, m, g, d), dtype=f64, device=dev), torch.zeros((b, m, g, d), dtype=f64, device=dev)
    reach = case["window"] or 1 << 40
    for x, (rows, cols) in enumerate(_lengths(case)):
        if rows == 0 or cols == 0:
            continue
        ahead = torch.arange(cols, device=dev) - (torch.arange(rows, device=dev)[:, None] + cols - rows)
        sees = (ahead > -reach) & (ahead <= 0 if case["causal"] else ahead < reach)
        some = sees.any(1)
        for y in range(h):
            q, k, v = s["q"][x, :rows, y].double(), s["k"][x, :cols, y * g // h].double(), s["v"][x, :cols, y * g // h].double()
            logit = torch.where(sees, (q * s["scale"]) @ k.t(), -math.inf)
            total = torch.logsumexp(logit, 1)
            p = torch.where(sees & some[:, None], torch.exp(logit - torch.where(some, total, 0.0)[:, None]), 0.0)
            o = p @ v
            if not back:
                out[x, :rows, y], lse[x, y, :rows] = o, total
                continue
            do = s["dout"][x, :rows, y].double()
            dv[x, :cols, y * g // h] += p.t() @ do
            # through the softmax: p * (dp - the row's mean of dp under p), that mean being do . o
            p *= do @ v.t() - torch.linalg.vecdot(do, o)[:, None]
            dq[x, :rows, y] = (p @ k) * s["scale"]
            dk[x, :cols, y * g // h] += (p.t() @ q) * s["scale"]
    return {"dq": dq, "dk": dk, "dv": dv} if back else {"out": out, "lse": lse}
