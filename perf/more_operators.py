"""Workloads of the operators that complete a block of the network and its
training: the projection with bias, activation and residual, the gated scan
(whole sequences with their gradients, and single tokens against a kept
state), and the orthogonalised update of a weight.

The sizes are the solver's own where there are any (10^6 unknowns, a 128 x 128
grid) and generic ones elsewhere.

``run`` computes the operators in elementary torch operations (``own`` false)
or through the library (``own`` true); ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-7
STEPS = 5
TRIPLE = (3.4445, -4.775, 2.0315)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the projection back from a feed-forward unit onto the residual stream, in a training step
        {"name": "linear_down_train", "op": "linear", "rows": 16384, "inner": 4096, "outer": 1024,
         "type": "bf16", "act": "none", "bias": False, "residual": True, "train": True},
        # a layer on the features of every unknown of the 1000 x 1000 grid, in a training step
        {"name": "linear_cells_train", "op": "linear", "rows": 1000000, "inner": 64, "outer": 64,
         "type": "fp32", "act": "silu", "bias": True, "residual": True, "train": True},
        # odd sizes that no tile divides, everything in the epilogue, in a training step
        {"name": "linear_odd_train", "op": "linear", "rows": 5000, "inner": 771, "outer": 1403,
         "type": "fp16", "act": "gelu", "bias": True, "residual": True, "train": True},
        # a few tokens: reading the weight is all the work
        {"name": "linear_few", "op": "linear", "rows": 4, "inner": 4096, "outer": 1024,
         "type": "bf16", "act": "none", "bias": True, "residual": True, "train": False},
        # training on four sequences of 4096 tokens
        {"name": "scan_train", "op": "scan", "seqs": 4, "total": 16384, "packed": False,
         "channels": 2048, "type": "bf16", "gate": "bf16", "train": True},
        # one very long sequence of few channels, evaluated once
        {"name": "scan_long", "op": "scan", "seqs": 1, "total": 131072, "packed": False,
         "channels": 256, "type": "fp16", "gate": "fp32", "train": False},
        # sequences of many lengths and an odd width in one call, in a training step
        {"name": "scan_packed_train", "op": "scan", "seqs": 23, "total": 12345, "packed": True,
         "channels": 999, "type": "fp32", "gate": "fp32", "train": True},
        # one sequence's next token: latency
        {"name": "step_one", "op": "step", "seqs": 1, "channels": 2048, "type": "bf16",
         "gate": "bf16"},
        # a server's batch of next tokens
        {"name": "step_many", "op": "step", "seqs": 2048, "channels": 4096, "type": "bf16",
         "gate": "bf16"},
        # the update of a wide weight
        {"name": "ortho_wide", "op": "ortho", "count": 1, "rows": 1024, "cols": 4096,
         "type": "bf16"},
        # a stack of a small network's weights: latency
        {"name": "ortho_small", "op": "ortho", "count": 12, "rows": 128, "cols": 64,
         "type": "fp32"},
        # a tall weight of odd sizes, in single precision
        {"name": "ortho_tall", "op": "ortho", "count": 1, "rows": 1403, "cols": 515,
         "type": "fp32"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A width: most real ones are multiples of 64."""
    n = _spread(rng, low, high)
    return max(low, n // 64 * 64) if n > 64 and rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "scan", "scan", "scan", "step", "ortho",
                     "ortho"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "linear":
        inner, outer = _width(rng, 16, 4096), _width(rng, 16, 4096)
        most = min((10 if kind == "fp32" else 64) * 10 ** 9 // (inner * outer),
                   64 * 10 ** 6 // max(inner, outer))
        return {"op": op, "rows": _spread(rng, 1, max(1, most)), "inner": inner, "outer": outer,
                "type": kind, "act": rng.choice(["none", "none", "silu", "gelu", "relu"]),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.6,
                "train": rng.random() < 0.6}
    if op == "ortho":
        rows, cols = _width(rng, 16, 4096), _width(rng, 16, 4096)
        if rows > 1024 and cols > 1024:  # the largest listed update is the dearest
            rows, cols = (1024, cols) if rng.random() < 0.5 else (rows, 1024)
        count = _spread(rng, 1, max(1, min(48, 2 ** 21 // (rows * cols))))
        return {"op": op, "count": count, "rows": rows, "cols": cols, "type": kind}
    gate = rng.choice([kind, "fp32"])
    if op == "step":
        channels = _width(rng, 16, 8192)
        return {"op": op, "seqs": _spread(rng, 1, max(1, 2 ** 23 // channels)),
                "channels": channels, "type": kind, "gate": gate}
    seqs = _spread(rng, 1, 64)
    channels = _width(rng, 16, 4096)
    total = seqs * _spread(rng, 1, max(1, min(131072, 2 ** 25 // (seqs * channels))))
    packed = rng.random() < 0.5
    if packed:
        total += rng.randrange(seqs)
    return {"op": op, "seqs": seqs, "total": total, "packed": packed, "channels": channels,
            "type": kind, "gate": gate, "train": rng.random() < 0.6}


def _lengths(case):
    """The lengths of a case's sequences: equal ones, or ragged ones that add up to its total."""
    n, total = case["seqs"], case["total"]
    if not case["packed"]:
        return [total // n] * n
    weight = [(5 * i * i + 2 * i + 3) % 13 for i in range(n)]
    weight[0] += 1
    edge = [total * sum(weight[:i]) // sum(weight) for i in range(n + 1)]
    return [b - a for a, b in zip(edge, edge[1:])]


def _size(kind):
    return 4 if kind == "fp32" else 2


def work(case):
    es = _size(case["type"])
    if case["op"] == "linear":
        m, k, n = case["rows"], case["inner"], case["outer"]
        few = n if case["bias"] else 0
        ends = (2 if case["residual"] else 1) * m * n
        if case["train"]:  # x, weight, bias, residual, dy; y and the gradients (the residual's is dy)
            return {"bytes": (2 * m * k + 2 * n * k + 2 * few + ends + m * n) * es,
                    "flops": 6 * m * n * k}
        return {"bytes": (m * k + n * k + few + ends) * es, "flops": 2 * m * n * k}
    if case["op"] == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        # the lower halves of A and of A^2, and the product with X
        step = m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n
        return {"bytes": 2 * case["count"] * m * n * es, "flops": case["count"] * STEPS * step}
    eg, c = _size(case["gate"]), case["channels"]
    tokens = case["seqs"] if case["op"] == "step" else case["total"]
    flow, states = tokens * c * (2 * es + eg), case["seqs"] * c * 8
    if case.get("train"):  # x, g, dh, both ends' states; h, dx, dg and theirs
        return {"bytes": 2 * (flow + states), "flops": 8 * tokens * c}
    return {"bytes": flow + states, "flops": 3 * tokens * c}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def leaf(t):
        return t.contiguous().requires_grad_(bool(case.get("train")))

    if case["op"] == "linear":
        m, k, n = case["rows"], case["inner"], case["outer"]
        s = {"case": case, "x": leaf(normal(m, k).to(kind)),
             "w": leaf((normal(n, k) / math.sqrt(k)).to(kind)),
             "b": leaf((0.3 * normal(n)).to(kind)) if case["bias"] else None,
             "r": leaf(normal(m, n).to(kind)) if case["residual"] else None}
        if case["train"]:
            s["dy"] = normal(m, n).to(kind)
        return s
    if case["op"] == "ortho":
        # a gradient: some strong directions above noise
        count, m, n = case["count"], case["rows"], case["cols"]
        rank = max(1, min(m, n) // 4)
        strong = normal(count, m, rank) * torch.linspace(1, 0.1, rank, device=dev)
        mat = torch.matmul(strong, normal(count, rank, n)) / math.sqrt(rank) + 0.2 * normal(
            count, m, n)
        return {"case": case, "m": (0.01 * mat).to(kind)}

    c, gate = case["channels"], TYPES[case["gate"]]
    if case["op"] == "step":
        lead = (case["seqs"],)
    elif case["packed"]:
        lead = (1, case["total"])
    else:
        lead = (case["seqs"], case["total"] // case["seqs"])
    # channels that forget within a token and ones that remember hundreds
    rate = torch.exp(1.0 - 7.0 * torch.rand(c, generator=gen, device=dev))
    g = -rate * torch.nn.functional.softplus(normal(*lead, c) + 1)
    s = {"case": case, "x": leaf(normal(*lead, c).to(kind)), "g": leaf(g.to(gate)),
         "s0": leaf(normal(case["seqs"], c)), "cu": None}
    if case["op"] == "step":
        return s
    s["lens"] = _lengths(case)
    if case["packed"]:
        edges = [0]
        for n in s["lens"]:
            edges.append(edges[-1] + n)
        s["cu"] = torch.tensor(edges, dtype=torch.int32, device=dev)
    if case["train"]:
        s["dh"] = normal(*lead, c).to(kind)
        s["ds"] = normal(case["seqs"], c)
    return s


# ---------------------------------------------------------------------------
# The operators, through the library or in elementary operations
# ---------------------------------------------------------------------------
def run(s):
    return (_library if own else _plain)(s)


def _library(s):
    import krylov_solvers_adjoint_amd as K
    case = s["case"]
    op, train = case["op"], case.get("train", False)
    if op == "linear":
        y = K.linear(s["x"], s["w"], s["b"], None if case["act"] == "none" else case["act"],
                     s["r"])
        if not train:
            return {"y": y}
        names = [n for n in ("x", "w", "b", "r") if s[n] is not None]
        grads = torch.autograd.grad(y, [s[n] for n in names], s["dy"])
        return {"y": y, **{"d" + n: t for n, t in zip(names, grads)}}
    if op == "ortho":
        return {"x": K.orthogonalise(s["m"], STEPS, TRIPLE, EPS)}
    if op == "step":
        return {"h": K.gated_scan_step(s["x"], s["g"], s["s0"]), "state": s["s0"]}
    h, state = K.gated_scan(s["x"], s["g"], initial_state=s["s0"], output_final_state=True,
                            cu_seqlens=s["cu"])
    if not train:
        return {"h": h, "state": state}
    dx, dg, ds0 = torch.autograd.grad((h, state), (s["x"], s["g"], s["s0"]), (s["dh"], s["ds"]))
    return {"h": h, "state": state, "dx": dx, "dg": dg, "ds0": ds0}


@torch.no_grad()
def _plain(s):
    return {"linear": _plain_linear, "ortho": _plain_ortho, "step": _plain_step,
            "scan": _plain_scan}[s["case"]["op"]](s)


def _activation(z, act):
    """The activation and its derivative (None: 1 everywhere)."""
    if act == "none":
        return z, None
    if act == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg * (1 + z * (1 - sg))
    if act == "gelu":
        half = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * half, half + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    on = (z > 0).to(z.dtype)
    return z * on, on


def _plain_linear(s):
    case, kind = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y, slope = _activation(z, case["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    if not case["train"]:
        return {"y": y.to(kind)}
    dz = s["dy"].float()
    if slope is not None:
        dz = dz * slope
    out = {"y": y.to(kind), "dx": (dz @ w).to(kind), "dw": (dz.t() @ x).to(kind)}
    if s["b"] is not None:
        out["db"] = dz.sum(0).to(kind)
    if s["r"] is not None:
        out["dr"] = s["dy"]
    return out


def _plain_ortho(s):
    a, b, c = TRIPLE
    x = s["m"].float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2).contiguous()
    x = x / (x.double().square().sum((-1, -2), keepdim=True).sqrt() + EPS).float()
    for _ in range(STEPS):
        gram = x @ x.transpose(-1, -2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(-1, -2).contiguous()
    return {"x": x.to(s["m"].dtype)}


def _plain_step(s):
    state = torch.exp(s["g"].float()) * s["s0"] + s["x"].float()
    s["s0"].copy_(state)
    return {"h": state.to(s["x"].dtype), "state": s["s0"]}


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, from zero: each turn joins spans twice as
    long."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], a[span:] * b[:-span] + b[span:]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _plain_scan(s):
    """All sequences as one: a decay of zero in front of each one's first token, whose input
    carries its initial state."""
    case, c = s["case"], s["case"]["channels"]
    dev = s["x"].device
    lens = torch.tensor(s["lens"], device=dev)
    end = torch.cumsum(lens, 0)
    some = lens > 0
    first, last = (end - lens)[some], (end - 1)[some]
    x, a = s["x"].float().reshape(-1, c), torch.exp(s["g"].float()).reshape(-1, c)
    s0 = s["s0"].detach()
    inner = a.clone()
    inner[first] = 0
    b = x.clone()
    b[first] += a[first] * s0[some]
    h = _doubling(inner, b)
    state = s0.clone()
    state[some] = h[last]
    out = {"h": h.reshape(s["x"].shape).to(s["x"].dtype), "state": state}
    if not case["train"]:
        return out
    dh = s["dh"].float().reshape(-1, c).clone()
    dh[last] += s["ds"][some]
    after = torch.cat([inner[1:], torch.zeros_like(inner[:1])])
    lam = torch.flip(_doubling(torch.flip(after, (0,)), torch.flip(dh, (0,))), (0,))
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = s0[some]
    ds0 = s["ds"].clone()
    ds0[some] = a[first] * lam[first]
    return {**out, "dx": lam.reshape(s["x"].shape).to(s["x"].dtype),
            "dg": (lam * a * before).reshape(s["g"].shape).to(s["g"].dtype), "ds0": ds0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
@torch.no_grad()
def exact(case, seed):
    s = prepare(case, seed)
    f = {n: t.detach().double() for n, t in s.items()
         if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if case["op"] == "linear":
        return _exact_linear(case, s, f)
    if case["op"] == "ortho":
        a, b, c = TRIPLE
        x = f["m"] / (torch.linalg.matrix_norm(f["m"])[:, None, None] + EPS)
        tall = case["rows"] > case["cols"]
        for _ in range(STEPS):
            xt = x.transpose(1, 2).contiguous()
            if tall:
                once = x.matmul(xt.matmul(x))
                twice = once.matmul(xt.matmul(x))
            else:
                once = x.matmul(xt).matmul(x)
                twice = x.matmul(xt).matmul(once)
            x = a * x + b * once + c * twice
        return {"x": x}
    if case["op"] == "step":
        state = f["x"] + f["g"].exp() * f["s0"]
        return {"h": state, "state": state}
    return _exact_scan(case, s, f)


def _exact_linear(case, s, f):
    z = f["x"] @ f["w"].t()
    if case["bias"]:
        z += f["b"]
    if case["act"] == "silu":
        e = torch.exp(-z)
        act, slope = z / (1 + e), (1 + e * (1 + z)) / (1 + e).square()
    elif case["act"] == "gelu":
        phi = torch.special.erfc(-z / math.sqrt(2)) / 2
        act, slope = z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif case["act"] == "relu":
        act, slope = torch.where(z > 0, z, 0), torch.where(z > 0, 1.0, 0.0).double()
    else:
        act, slope = z, torch.ones_like(z)
    if case["residual"]:
        act = act + f["r"]
    if not case["train"]:
        return {"y": act}
    dz = f["dy"] * slope
    out = {"y": act, "dx": dz @ f["w"], "dw": dz.t() @ f["x"]}
    if case["bias"]:
        out["db"] = dz.sum(0)
    if case["residual"]:
        out["dr"] = f["dy"]
    return out


def _exact_scan(case, s, f):
    """Token by token, all sequences side by side, the longest first."""
    c, dev = case["channels"], s["x"].device
    lens = torch.tensor(s["lens"])
    order = torch.argsort(lens, descending=True, stable=True)
    begin = (torch.cumsum(lens, 0) - lens)[order].to(dev)
    longest = max(s["lens"])
    live = (lens[None] > torch.arange(longest)[:, None]).sum(1).tolist()  # that have a token t
    order = order.to(dev)
    x, a = f["x"].reshape(-1, c), f["g"].exp().reshape(-1, c)
    h, state, before = torch.empty_like(x), f["s0"][order], f["s0"][order]
    for t, n in enumerate(live):
        at = begin[:n] + t
        state[:n] = a[at] * state[:n] + x[at]
        h[at] = state[:n]
    out = {"h": h.reshape(s["x"].shape), "state": torch.empty_like(state).index_copy_(0, order,
                                                                                     state)}
    if not case["train"]:
        return out
    dh = f["dh"].reshape(-1, c)
    lam, dg, carried = torch.empty_like(x), torch.empty_like(x), f["ds"][order]
    for t in reversed(range(longest)):
        at = begin[:live[t]] + t
        now = dh[at] + carried[:live[t]]
        lam[at] = now
        now = now * a[at]
        carried[:live[t]] = now
        dg[at] = now * (h[at - 1] if t else before[:live[t]])
    return {**out, "dx": lam.reshape(s["x"].shape), "dg": dg.reshape(s["g"].shape),
            "ds0": torch.empty_like(carried).index_copy_(0, order, carried)}
