"""Workloads of the network operators that stand next to the solver: layer
norm, the gated feed-forward unit and the gated delta rule (whole sequences
with their gradients, and single tokens against a kept state).

A network that predicts a system's coefficients from per-unknown features is
a stack of these three, trained through the solver's adjoint.  The cases take
the solver's own sizes where there are any (10^6 unknowns, a 128 x 128 grid)
and generic ones elsewhere.

``run`` computes the operators in elementary torch operations (``own`` false)
or through the library (``own`` true); ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
CHUNK = 64
EPS = 1e-5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one feature row for every unknown of the 1000 x 1000 grid, in a training step
        {"name": "norm_cells_train", "op": "norm", "rows": 1000000, "cols": 64, "type": "fp32",
         "train": True},
        # the unknowns of a 128 x 128 grid as wide tokens, in a training step
        {"name": "norm_tokens_train", "op": "norm", "rows": 16384, "cols": 1024, "type": "bf16",
         "train": True},
        # a few odd rows: launch latency and the reduction of the weight's gradient
        {"name": "norm_few_train", "op": "norm", "rows": 37, "cols": 1111, "type": "fp16",
         "train": True},
        # the feed-forward unit of a 128 x 128 grid's tokens, in a training step
        {"name": "ffn_train", "op": "ffn", "rows": 16384, "inner": 1024, "outer": 4096,
         "type": "bf16", "act": "silu", "train": True},
        # a wide unit evaluated once for many tokens
        {"name": "ffn_wide", "op": "ffn", "rows": 8192, "inner": 2048, "outer": 8192,
         "type": "bf16", "act": "gelu", "train": False},
        # a few tokens: reading the weights is all the work
        {"name": "ffn_few", "op": "ffn", "rows": 4, "inner": 1024, "outer": 4096,
         "type": "bf16", "act": "silu", "train": False},
        # odd sizes that no tile divides, in single precision, in a training step
        {"name": "ffn_odd_train", "op": "ffn", "rows": 1000, "inner": 515, "outer": 1403,
         "type": "fp32", "act": "silu", "train": True},
        # training on four sequences of 4096 tokens
        {"name": "delta_train", "op": "delta", "seqs": 4, "total": 16384, "packed": False,
         "kheads": 16, "vheads": 16, "dk": 128, "dv": 128, "type": "bf16", "train": True},
        # sequences of many lengths in one call, carried on from kept states
        {"name": "delta_packed", "op": "delta", "seqs": 12, "total": 9001, "packed": True,
         "kheads": 4, "vheads": 8, "dk": 64, "dv": 128, "type": "fp16", "train": False},
        # small, odd, shared heads, single precision, in a training step
        {"name": "delta_odd_train", "op": "delta", "seqs": 2, "total": 666, "packed": False,
         "kheads": 3, "vheads": 6, "dk": 48, "dv": 80, "type": "fp32", "train": True},
        # one sequence's next token: latency
        {"name": "step_one", "op": "step", "seqs": 1, "kheads": 8, "vheads": 16, "dk": 128,
         "dv": 128, "type": "bf16"},
        # a server's batch of next tokens
        {"name": "step_many", "op": "step", "seqs": 128, "kheads": 16, "vheads": 32, "dk": 128,
         "dv": 128, "type": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "ffn", "ffn", "delta", "delta", "step"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        cols = _spread(rng, 32, 8192)
        return {"op": op, "rows": _spread(rng, 1, 50000000 // cols), "cols": cols, "type": kind,
                "train": rng.random() < 0.7}
    if op == "ffn":
        inner, outer = _spread(rng, 64, 2048), _spread(rng, 64, 8192)
        if rng.random() < 0.6:  # most real widths are multiples of 64
            inner, outer = max(64, inner // 64 * 64), max(64, outer // 64 * 64)
        most = (4 if kind == "fp32" else 32) * 10 ** 9 // (inner * outer)
        return {"op": op, "rows": _spread(rng, 1, max(1, min(16384, most))), "inner": inner,
                "outer": outer, "type": kind, "act": rng.choice(["silu", "gelu", "relu"]),
                "train": rng.random() < 0.6}
    shared = rng.choice([1, 1, 2, 4])
    kheads = _spread(rng, 1, 8)
    vheads = kheads * shared
    size = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64), None])
    dk, dv = size or (_spread(rng, 16, 128), _spread(rng, 16, 128))
    if op == "step":
        return {"op": op, "seqs": _spread(rng, 1, 128), "kheads": kheads, "vheads": vheads,
                "dk": dk, "dv": dv, "type": kind}
    seqs = _spread(rng, 1, 12)
    packed = rng.random() < 0.5
    total = seqs * _spread(rng, 1, max(1, min(4096, 120000 // (seqs * vheads))))
    if packed:
        total += rng.randrange(seqs)
    return {"op": op, "seqs": seqs, "total": total, "packed": packed, "kheads": kheads,
            "vheads": vheads, "dk": dk, "dv": dv, "type": kind, "train": rng.random() < 0.6}


def _lengths(case):
    """The lengths of a case's sequences: equal ones, or ragged ones that add up to its total."""
    n, total = case["seqs"], case["total"]
    if not case["packed"]:
        return [total // n] * n
    weight = [1 + (7 * i * i + 3 * i) % 11 for i in range(n)]
    edge = [total * sum(weight[:i]) // sum(weight) for i in range(n + 1)]
    return [b - a for a, b in zip(edge, edge[1:])]


def work(case):
    es = 4 if case["type"] == "fp32" else 2
    if case["op"] == "norm":
        size = case["rows"] * case["cols"]
        arrays, rows = (4, 4) if case["train"] else (2, 2)
        return {"bytes": (arrays * size + rows * case["cols"]) * es,
                "flops": size * (19 if case["train"] else 8)}
    if case["op"] == "ffn":
        m, k, f = case["rows"], case["inner"], case["outer"]
        if case["train"]:  # x, dh, both weights; h, dx and both weights' gradients
            return {"bytes": (2 * m * k + 2 * m * f + 4 * k * f) * es, "flops": 12 * m * k * f}
        return {"bytes": (m * k + m * f + 2 * k * f) * es, "flops": 4 * m * k * f}
    hk, hv, dk, dv = case["kheads"], case["vheads"], case["dk"], case["dv"]
    state = case["seqs"] * hv * dk * dv * 4
    tokens = case["seqs"] if case["op"] == "step" else case["total"]
    qkvo = tokens * (2 * hk * dk + 2 * hv * dv) * es
    gates = tokens * hv * 8
    # the recurrence itself: S^T k, the update and S^T q, two operations each
    step = tokens * hv * dk * dv * 7
    if case["op"] == "step" or not case["train"]:
        return {"bytes": qkvo + gates + 2 * state, "flops": step}
    # o and every input's gradient out; do and the final state's gradient in
    return {"bytes": 2 * (qkvo + gates) + 4 * state, "flops": 3 * step}


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

    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        x = normal(rows, cols) * (0.5 + normal(rows, 1).abs()) + normal(rows, 1)
        return {"case": case, "x": leaf(x.to(kind)), "w": leaf((1 + 0.1 * normal(cols)).to(kind)),
                "b": leaf((0.1 * normal(cols)).to(kind)), "dy": normal(rows, cols).to(kind)}
    if case["op"] == "ffn":
        m, k, f = case["rows"], case["inner"], case["outer"]
        s = {"case": case, "x": leaf(normal(m, k).to(kind)),
             "wg": leaf((normal(f, k) / math.sqrt(k)).to(kind)),
             "wu": leaf((normal(f, k) / math.sqrt(k)).to(kind))}
        if case["train"]:
            s["dh"] = normal(m, f).to(kind)
        return s

    hk, hv, dk, dv = case["kheads"], case["vheads"], case["dk"], case["dv"]
    step = case["op"] == "step"
    if step:
        lead = (case["seqs"],)
    elif case["packed"]:
        lead = (1, case["total"])
    else:
        lead = (case["seqs"], case["total"] // case["seqs"])

    def unit(t):
        return t / t.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)

    # keys that repeat themselves in part, as neighbouring tokens' do
    k = unit(normal(*lead, hk, dk) + 0.5 * normal(*([1] * len(lead)), hk, dk))
    rate = torch.exp(-1.0 - 4.0 * torch.rand(hv, generator=gen, device=dev))
    g = -rate * torch.nn.functional.softplus(normal(*lead, hv) + 1)
    s = {"case": case, "q": leaf(unit(normal(*lead, hk, dk)).to(kind)), "k": leaf(k.to(kind)),
         "v": leaf(normal(*lead, hv, dv).to(kind)), "g": leaf(g),
         "beta": leaf(torch.sigmoid(normal(*lead, hv))),
         "s0": leaf(normal(case["seqs"], hv, dk, dv) / math.sqrt(dk)), "cu": None}
    if not step:
        s["lens"] = _lengths(case)
        if case["packed"]:
            edges = [0]
            for n in s["lens"]:
                edges.append(edges[-1] + n)
            s["cu"] = torch.tensor(edges, dtype=torch.int32, device=dev)
        if case["train"]:
            s["do"] = normal(*lead, hv, dv).to(kind)
            s["ds"] = normal(case["seqs"], hv, dk, dv) / math.sqrt(dk)
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
    if op == "norm":
        y = K.layer_norm(s["x"], s["w"], s["b"], EPS)
        if not train:
            return {"y": y}
        dx, dw, db = torch.autograd.grad(y, (s["x"], s["w"], s["b"]), s["dy"])
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    if op == "ffn":
        h = K.gated_ffn(s["x"], s["wg"], s["wu"], case["act"])
        if not train:
            return {"h": h}
        dx, dwg, dwu = torch.autograd.grad(h, (s["x"], s["wg"], s["wu"]), s["dh"])
        return {"h": h, "dx": dx, "dwg": dwg, "dwu": dwu}
    if op == "step":
        o = K.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"])
        return {"o": o, "state": s["s0"]}
    o, state = K.gated_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"],
                                  initial_state=s["s0"], output_final_state=True,
                                  cu_seqlens=s["cu"])
    if not train:
        return {"o": o, "state": state}
    names = ("q", "k", "v", "g", "beta", "s0")
    grads = torch.autograd.grad((o, state), [s[n] for n in names], (s["do"], s["ds"]))
    return {"o": o, "state": state, **{"d" + n: t for n, t in zip(names, grads)}}


@torch.no_grad()
def _plain(s):
    op = s["case"]["op"]
    return {"norm": _plain_norm, "ffn": _plain_ffn, "step": _plain_step,
            "delta": _plain_delta}[op](s)


def _plain_norm(s):
    kind = s["x"].dtype
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    xc = x - x.mean(-1, keepdim=True)
    rstd = (xc.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = xc * rstd
    y = (n * w + b).to(kind)
    if not s["case"]["train"]:
        return {"y": y}
    dy = s["dy"].float()
    t = dy * w
    dx = rstd * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(kind), "dw": (dy * n).sum(0).to(kind), "db": dy.sum(0).to(kind)}


def _activation(a, act):
    """The activation and its derivative."""
    if act == "silu":
        sg = torch.sigmoid(a)
        return a * sg, sg * (1 + a * (1 - sg))
    if act == "gelu":
        half = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * half, half + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    on = (a > 0).to(a.dtype)
    return a * on, on


def _plain_ffn(s):
    kind = s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    a, b = x @ wg.t(), x @ wu.t()
    f, df = _activation(a, s["case"]["act"])
    h = (f * b).to(kind)
    if not s["case"]["train"]:
        return {"h": h}
    dh = s["dh"].float()
    da, db = dh * b * df, dh * f
    return {"h": h, "dx": (da @ wg + db @ wu).to(kind), "dwg": (da.t() @ x).to(kind),
            "dwu": (db.t() @ x).to(kind)}


def _plain_step(s):
    case = s["case"]
    kind, group = s["q"].dtype, case["vheads"] // case["kheads"]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    S = s["s0"] * torch.exp(s["g"])[..., None, None]
    m = s["v"].float() - (S * k[..., None]).sum(-2)
    S = S + k[..., None] * (s["beta"][..., None] * m)[..., None, :]
    s["s0"].copy_(S)
    o = (S * q[..., None]).sum(-2) / math.sqrt(case["dk"])
    return {"o": o.to(kind), "state": s["s0"]}


def _places(lens, block, dev):
    """Where each place of the padded sequences [N, T] comes from in the packed tokens, whether
    it is a token, and each token's place among the padded ones."""
    long = max(1, -(-max(lens) // block)) * block
    place = torch.arange(long, device=dev)
    n = torch.tensor(lens, device=dev)
    start = torch.cumsum(n, 0) - n
    real = place[None] < n[:, None]
    source = torch.where(real, start[:, None] + place[None], 0)
    return source, real, real.reshape(-1).nonzero().squeeze(1)


def _plain_delta(s):
    """In chunks of 64 tokens: inside a chunk the updates solve one unit lower triangular system,
    from chunk to chunk the state is carried."""
    case = s["case"]
    kind, hk, hv = s["q"].dtype, case["kheads"], case["vheads"]
    dk, dv, nseq, group = case["dk"], case["dv"], case["seqs"], case["vheads"] // case["kheads"]
    scale = 1 / math.sqrt(dk)
    dev = s["q"].device
    source, real, back = _places(s["lens"], CHUNK, dev)
    nc = source.shape[1] // CHUNK

    def chunks(t, width):
        """[.., H, width] of the tokens -> [chunk, N, H, CHUNK, width]"""
        t = t.reshape(-1, *t.shape[2:]).float()
        t = t.reshape(t.shape[0], t.shape[1], -1)[source.reshape(-1)]
        t = t * real.reshape(-1, 1, 1)
        return t.reshape(nseq, nc, CHUNK, -1, width).permute(1, 0, 3, 2, 4).contiguous()

    def tokens(t, like):
        """... and back, in the layout of `like`"""
        t = t.permute(1, 0, 3, 2, 4).reshape(nseq * nc * CHUNK, -1)[back]
        return t.reshape(like.shape).to(like.dtype)

    q = chunks(s["q"], dk).repeat_interleave(group, 2)
    k = chunks(s["k"], dk).repeat_interleave(group, 2)
    v, g, beta = chunks(s["v"], dv), chunks(s["g"], 1), chunks(s["beta"], 1)
    G = torch.cumsum(g.double(), -2)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp(torch.where(low, G - G.transpose(-1, -2), -torch.inf)).float()
    eG, eC, eL = torch.exp(G).float(), torch.exp(G[..., -1:, :] - G).float(), \
        torch.exp(G[..., -1:, :]).float()
    kt = k.transpose(-1, -2).contiguous()
    Abar = decay.tril(-1) * (k @ kt)
    A = beta * Abar
    T = torch.eye(CHUNK, device=dev).expand(A.shape).contiguous()
    for i in range(1, CHUNK):  # forward substitution of (I + A) T = I
        T[..., i, :i] = -(A[..., i, :i, None] * T[..., :i, :i]).sum(-2)
    P = scale * decay * (q @ kt)
    S = s["s0"].detach().clone()
    states, news, outs = [], [], []
    for c in range(nc):
        R = v[c] - eG[c] * (k[c] @ S)
        N = T[c] @ (beta[c] * R)
        outs.append(scale * eG[c] * (q[c] @ S) + P[c] @ N)
        states.append(S)
        news.append(N)
        S = eL[c] * S + (k[c] * eC[c]).transpose(-1, -2).contiguous() @ N
    o = tokens(torch.stack(outs), s["v"])
    if not case["train"]:
        return {"o": o, "state": S}

    do = chunks(s["do"], dv)
    S0, N = torch.stack(states), torch.stack(news)
    Pt, Tt = P.transpose(-1, -2).contiguous(), T.transpose(-1, -2).contiguous()
    qs = (scale * eG * q).transpose(-1, -2).contiguous()
    kg = (eG * k).transpose(-1, -2).contiguous()
    dS = s["ds"]
    ends, solved = [None] * nc, [None] * nc
    for c in reversed(range(nc)):
        X = Tt[c] @ (Pt[c] @ do[c] + eC[c] * (k[c] @ dS))  # the adjoint system
        ends[c], solved[c] = dS, X
        dS = eL[c] * dS + qs[c] @ do[c] - kg[c] @ (beta[c] * X)
    X, dSC = torch.stack(solved), torch.stack(ends)
    dR = beta * X
    S0t, Nt = S0.transpose(-1, -2).contiguous(), N.transpose(-1, -2).contiguous()
    dP = scale * decay * (do @ Nt)
    dA = decay.tril(-1) * (X @ Nt)  # of -Abar, before beta
    KS = k @ S0
    dq = scale * eG * (do @ S0t) + dP @ k
    into = -eG * (dR @ S0t) - (beta * dA) @ k
    away = dP.transpose(-1, -2).contiguous() @ q - (beta * dA).transpose(-1, -2).contiguous() @ k \
        + eC * (N @ dSC.transpose(-1, -2).contiguous())
    dbeta = (X * (v - eG * KS)).sum(-1, keepdim=True) - (dA * (k @ kt)).sum(-1, keepdim=True)
    SC = eL * S0 + (k * eC).transpose(-1, -2).contiguous() @ N
    dG = ((q * dq).sum(-1, keepdim=True) + (k * (into - away)).sum(-1, keepdim=True)).double()
    dG[..., -1, 0] += (SC * dSC).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dG, (-2,)), -2), (-2,)).float()

    def shared(t):
        return t.reshape(nc, nseq, hk, group, CHUNK, dk).sum(3)

    return {"o": o, "state": S, "dq": tokens(shared(dq), s["q"]),
            "dk": tokens(shared(into + away), s["k"]), "dv": tokens(dR, s["v"]),
            "dg": tokens(dg, s["g"]), "dbeta": tokens(dbeta, s["beta"]), "ds0": dS}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
@torch.no_grad()
def exact(case, seed):
    s = prepare(case, seed)
    f = {n: t.detach().double() for n, t in s.items()
         if isinstance(t, torch.Tensor) and t.is_floating_point()}
    if case["op"] == "norm":
        x = f["x"]
        mean = x.mean(1, keepdim=True)
        sd = ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
        n = (x - mean) / sd
        y = n * f["w"] + f["b"]
        if not case["train"]:
            return {"y": y}
        u = f["dy"] * f["w"]
        cols = case["cols"]
        dx = (u - u.sum(1, keepdim=True) / cols - n * ((u * n).sum(1, keepdim=True) / cols)) / sd
        return {"y": y, "dx": dx, "dw": (f["dy"] * n).sum(0), "db": f["dy"].sum(0)}
    if case["op"] == "ffn":
        a, b = f["x"] @ f["wg"].t(), f["x"] @ f["wu"].t()
        if case["act"] == "silu":
            act = a / (1 + torch.exp(-a))
            slope = (1 + torch.exp(-a) * (1 + a)) / (1 + torch.exp(-a)).square()
        elif case["act"] == "gelu":
            act = 0.5 * a * torch.special.erfc(-a / math.sqrt(2))
            slope = 0.5 * torch.special.erfc(-a / math.sqrt(2)) \
                + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        else:
            act, slope = torch.where(a > 0, a, 0), torch.where(a > 0, 1.0, 0.0).double()
        if not case["train"]:
            return {"h": act * b}
        da, db = f["dh"] * b * slope, f["dh"] * act
        return {"h": act * b, "dx": da @ f["wg"] + db @ f["wu"], "dwg": da.t() @ f["x"],
                "dwu": db.t() @ f["x"]}
    return _exact_step(case, f) if case["op"] == "step" else _exact_delta(case, s, f)


def _exact_step(case, f):
    group = case["vheads"] // case["kheads"]
    q, k = (f[n].repeat_interleave(group, 1) for n in ("q", "k"))
    S = f["s0"] * f["g"].exp()[:, :, None, None]
    m = f["v"] - torch.matmul(k[:, :, None], S)[:, :, 0]
    S = S + k[:, :, :, None] * (f["beta"][:, :, None] * m)[:, :, None, :]
    return {"o": torch.matmul(q[:, :, None], S)[:, :, 0] * case["dk"] ** -0.5, "state": S}


def _exact_delta(case, s, f):
    """Token by token; the gradients by the reverse of each token's step."""
    hk, hv, dk, dv = case["kheads"], case["vheads"], case["dk"], case["dv"]
    group, scale, nseq = hv // hk, dk ** -0.5, case["seqs"]
    block = 64
    source, real, back = _places(s["lens"], block, s["q"].device)
    long = source.shape[1]

    def steps(t, heads):
        t = t.reshape(-1, *t.shape[2:])[source.reshape(-1)] * \
            real.reshape(-1, *([1] * (t.dim() - 2)))
        t = t.reshape(nseq, long, *t.shape[1:]).transpose(0, 1)
        return t.repeat_interleave(group, 2) if heads == hk and group > 1 else t

    q, k, v = steps(f["q"], hk), steps(f["k"], hk), steps(f["v"], hv)
    if group == 1:
        g, beta = steps(f["g"], hv), steps(f["beta"], hv)
    else:
        g, beta = steps(f["g"], -1), steps(f["beta"], -1)
    a = g.exp()

    def step(S, t):
        """(decayed state, error of the prediction, state after the token)"""
        D = S * a[t][:, :, None, None]
        m = v[t] - torch.matmul(k[t][:, :, None], D)[:, :, 0]
        return D, m, D + k[t][:, :, :, None] * (beta[t][:, :, None] * m)[:, :, None, :]

    def tokens(seq, like):
        return seq.transpose(0, 1).reshape(nseq * long, -1)[back].reshape(like.shape)

    S, kept, o = f["s0"], [], torch.empty_like(v)
    for t in range(long):
        if t % block == 0:
            kept.append(S)
        S = step(S, t)[2]
        o[t] = scale * torch.matmul(q[t][:, :, None], S)[:, :, 0]
    out = {"o": tokens(o, s["v"]), "state": S}
    if not case["train"]:
        return out
    do = steps(f["do"], hv) if group == 1 else steps(f["do"], -1)
    dS = f["ds"]
    dq, dk_, dv_ = (torch.empty_like(t) for t in (q, k, v))
    dg, dbeta = torch.empty_like(g), torch.empty_like(g)
    for c in reversed(range(long // block)):
        S, seen = kept[c], []
        for t in range(c * block, (c + 1) * block):
            D, m, S = step(S, t)
            seen.append((D, m, S))
        for t in reversed(range(c * block, (c + 1) * block)):
            D, m, after = seen.pop()
            dS = dS + scale * q[t][:, :, :, None] * do[t][:, :, None, :]
            dq[t] = scale * torch.matmul(after, do[t][..., None])[..., 0]
            bm = beta[t][:, :, None] * m
            dn = torch.matmul(k[t][:, :, None], dS)[:, :, 0]
            dbeta[t] = (dn * m).sum(-1)
            dm = beta[t][:, :, None] * dn
            dv_[t] = dm
            dk_[t] = torch.matmul(dS, bm[..., None])[..., 0] - \
                torch.matmul(D, dm[..., None])[..., 0]
            dD = dS - k[t][:, :, :, None] * dm[:, :, None, :]
            dg[t] = (dD * D).sum((-1, -2))
            dS = dD * a[t][:, :, None, None]

    def shared(t):
        return t.reshape(long, nseq, hk, group, dk).sum(3)

    return {**out, "dq": tokens(shared(dq), s["q"]), "dk": tokens(shared(dk_), s["k"]),
            "dv": tokens(dv_, s["v"]), "dg": tokens(dg, s["g"]),
            "dbeta": tokens(dbeta, s["beta"]), "ds0": dS}
