"""Plain 64-bit forms of the network operators (token by token, element by
element) and the error bounds their tests use."""
from __future__ import annotations

import math

import torch

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24          # half a step of fp32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def gen(seed: int) -> torch.Generator:
    return torch.Generator().manual_seed(seed)


def layer_norm(x, w, b, eps):
    mean = x.mean(-1, keepdim=True)
    var = (x - mean).square().mean(-1, keepdim=True)
    y = (x - mean) / (var + eps).sqrt()
    y = y if w is None else y * w
    return y if b is None else y + b


def activation(a, act):
    if act == "silu":
        return a * torch.sigmoid(a)
    if act == "gelu":
        return a * torch.special.erfc(-a / math.sqrt(2)) / 2
    return torch.where(a > 0, a, torch.zeros_like(a))


def gated_ffn(x, wg, wu, act):
    return activation(x @ wg.t(), act) * (x @ wu.t())


def delta_sequence(q, k, v, g, beta, s0, scale):
    """One sequence: q, k [T, Hk, dk], v [T, Hv, dv], g, beta [T, Hv], s0 [Hv, dk, dv]."""
    group = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    S, out = s0, []
    for t in range(v.shape[0]):
        S = g[t].exp()[:, None, None] * S
        m = v[t] - (S * k[t][:, :, None]).sum(1)
        S = S + k[t][:, :, None] * (beta[t][:, None] * m)[:, None, :]
        out.append(scale * (S * q[t][:, :, None]).sum(1))
    o = torch.stack(out) if out else v.new_zeros(v.shape)
    return o, S


def delta_rule(q, k, v, g, beta, s0, scale, edges=None):
    """Batched [B, T, ...], or one row of sequences between the edges."""
    if edges is None:
        parts = [delta_sequence(*(t[i] for t in (q, k, v, g, beta, s0)), scale)
                 for i in range(q.shape[0])]
        return torch.stack([o for o, _ in parts]), torch.stack([s for _, s in parts])
    outs = [v.new_zeros(edges[0], *v.shape[2:])]
    states = []
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        o, s = delta_sequence(*(t[0, a:b] for t in (q, k, v, g, beta)), s0[i], scale)
        outs.append(o)
        states.append(s)
    outs.append(v.new_zeros(v.shape[1] - edges[-1], *v.shape[2:]))
    return torch.cat(outs)[None], torch.stack(states)


def rel(got, want) -> float:
    """2-norm of the difference over the 2-norm of `want` (or of the difference, if that is 0)."""
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    n = want.norm().item()
    d = (got - want).norm().item()
    return d / n if n else d
