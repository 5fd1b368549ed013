"""Learning a diffusion coefficient through the solver's adjoint.

A small network reads five features of every unknown of an N x N grid and
predicts a log conductivity; the conductances of the grid's edges, the matrix
and its solution follow, and the loss compares that solution with the one of
the hidden conductivity.  One step's gradient runs through the adjoint solve,
the matrix's values and the network:

    features -> projection -> [layer norm -> gated delta rule along each grid
    line -> residual] -> [layer norm -> gated feed-forward unit -> residual]
    -> layer norm -> head -> conductivity -> A(c) x = b -> loss

``step_by_step`` evaluates the same network token by token along the lines
with ``gated_delta_step``, as a program does that meets its unknowns one at a
time.

``ScanNetwork`` is the lighter one: a gated scan along the lines in place of the
delta rule, and every projection with its bias, activation and residual in one
call (``linear``).  ``Orthogonalised`` is an optimiser for either: a weight
matrix moves by its orthogonalised momentum (``orthogonalise``), everything else
as Adam says.

    python examples/coefficient_network.py [--grid 32] [--steps 40]
        [--mixer delta|scan] [--optimizer adam|orthogonal]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import krylov_solvers_adjoint_amd as K  # noqa: E402
import workloads as W  # noqa: E402


class Network(torch.nn.Module):
    """Five features of each unknown [lines, unknowns, 5] -> log conductivity."""

    def __init__(self, width=64, heads=2, size=32, inner=128, dtype=torch.float32):
        super().__init__()
        self.heads, self.size, self.dtype = heads, size, dtype

        def param(*shape, scale=None):
            s = shape[-1] ** -0.5 if scale is None else scale
            return torch.nn.Parameter(s * torch.randn(*shape))

        def norm():
            return torch.nn.ParameterList([torch.ones(width), torch.zeros(width)])
        self.enter = param(width, 5)
        self.norms = torch.nn.ModuleList([norm() for _ in range(3)])
        self.qkv = param(3 * heads * size, width)
        self.gates = param(2 * heads, width)
        self.mix = param(width, heads * size)
        self.w_gate, self.w_up, self.w_down = param(inner, width), param(inner, width), \
            param(width, inner)
        self.head = param(1, width, scale=0.02)

    def _token_inputs(self, h):
        """q, k, v [.., heads, size] (unit q and k) and the gates of the tokens h [.., width]."""
        n = K.layer_norm(h, *self.norms[0])
        q, k, v = (n @ self.qkv.t()).unflatten(-1, (3, self.heads, self.size)).unbind(-3)
        q, k = (t / t.square().sum(-1, keepdim=True).add(1e-6).sqrt() for t in (q, k))
        g, beta = (n @ self.gates.t()).float().unflatten(-1, (2, self.heads)).unbind(-2)
        return (q.to(self.dtype), k.to(self.dtype), v.to(self.dtype),
                -torch.nn.functional.softplus(g), torch.sigmoid(beta))

    def _finish(self, h, o):
        h = h + o.flatten(-2).float() @ self.mix.t()
        n = K.layer_norm(h, *self.norms[1]).to(self.dtype)
        f = K.gated_ffn(n, self.w_gate.to(self.dtype), self.w_up.to(self.dtype))
        h = h + f.float() @ self.w_down.t()
        return (K.layer_norm(h, *self.norms[2]) @ self.head.t())[..., 0]

    def forward(self, features):
        h = features @ self.enter.t()
        o, _ = K.gated_delta_rule(*self._token_inputs(h))
        return self._finish(h, o)

    @torch.no_grad()
    def step_by_step(self, features):
        """The same, one unknown of every line at a time against kept states."""
        lines, length, _ = features.shape
        state = torch.zeros(lines, self.heads, self.size, self.size, device=features.device)
        out = []
        for t in range(length):
            h = features[:, t] @ self.enter.t()
            out.append(self._finish(h, K.gated_delta_step(*self._token_inputs(h), state)))
        return torch.stack(out, 1)


class ScanNetwork(torch.nn.Module):
    """The same features and output through gated scans and projections with epilogues."""

    def __init__(self, width=64, inner=128, dtype=torch.float32):
        super().__init__()
        self.width, self.dtype = width, dtype

        def param(*shape, scale=None):
            s = shape[-1] ** -0.5 if scale is None else scale
            return torch.nn.Parameter(s * torch.randn(*shape))

        def norm():
            return torch.nn.ParameterList([torch.ones(width), torch.zeros(width)])
        self.enter, self.enter_bias = param(width, 5), torch.nn.Parameter(torch.zeros(width))
        self.norms = torch.nn.ModuleList([norm() for _ in range(3)])
        self.value, self.gate, self.mix = param(width, width), param(width, width), \
            param(width, width)
        # channels that remember from one unknown to a hundred
        self.gate_bias = torch.nn.Parameter(torch.linspace(1.0, -5.0, width))
        self.w_gate, self.w_up, self.w_down = param(inner, width), param(inner, width), \
            param(width, inner)
        self.head, self.head_bias = param(1, width, scale=0.02), torch.nn.Parameter(torch.zeros(1))

    def _enter(self, features):
        return K.linear(features.to(self.dtype), self.enter.to(self.dtype), self.enter_bias, "gelu")

    def _scan_inputs(self, h):
        """What the scan takes in and its log decays, of the tokens h [.., width]."""
        n = K.layer_norm(h, *self.norms[0])
        g = K.linear(n, self.gate.to(self.dtype), self.gate_bias)
        return K.linear(n, self.value.to(self.dtype)), -torch.nn.functional.softplus(g)

    def _finish(self, h, o):
        h = K.linear(o, self.mix.to(self.dtype), residual=h)
        n = K.layer_norm(h, *self.norms[1])
        f = K.gated_ffn(n, self.w_gate.to(self.dtype), self.w_up.to(self.dtype))
        h = K.linear(f, self.w_down.to(self.dtype), residual=h)
        return K.linear(K.layer_norm(h, *self.norms[2]), self.head.to(self.dtype),
                        self.head_bias)[..., 0].float()

    def forward(self, features):
        h = self._enter(features)
        o, _ = K.gated_scan(*self._scan_inputs(h))
        return self._finish(h, o)

    @torch.no_grad()
    def step_by_step(self, features):
        """The same, one unknown of every line at a time against kept states."""
        lines, length, _ = features.shape
        state = torch.zeros(lines, self.width, device=features.device)
        out = []
        for t in range(length):
            h = self._enter(features[:, t])
            out.append(self._finish(h, K.gated_scan_step(*self._scan_inputs(h), state)))
        return torch.stack(out, 1)


class Orthogonalised(torch.optim.Optimizer):
    """A matrix with at least `least` rows and columns moves by its momentum
    orthogonalised, so that every direction moves alike; the other parameters by
    Adam."""

    def __init__(self, params, lr=5e-3, momentum=0.9, least=8, betas=(0.9, 0.999), eps=1e-8):
        super().__init__(params, dict(lr=lr, momentum=momentum, least=least, betas=betas, eps=eps))

    @torch.no_grad()
    def step(self):
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                s = self.state[p]
                if p.dim() == 2 and min(p.shape) >= group["least"]:
                    m = s.setdefault("momentum", torch.zeros_like(p))
                    m.mul_(group["momentum"]).add_(p.grad)
                    update = K.orthogonalise(p.grad + group["momentum"] * m)
                    p.add_(update, alpha=-group["lr"] * max(1, p.shape[0] / p.shape[1]) ** 0.5)
                    continue
                b1, b2 = group["betas"]
                if not s:
                    s.update(t=0, m=torch.zeros_like(p), v=torch.zeros_like(p))
                s["t"] += 1
                s["m"].lerp_(p.grad, 1 - b1)
                s["v"].lerp_(p.grad.square(), 1 - b2)
                root = (s["v"] / (1 - b2 ** s["t"])).sqrt_().add_(group["eps"])
                p.addcdiv_(s["m"], root, value=-group["lr"] / (1 - b1 ** s["t"]))


class Diffusion:
    """A(c) x = b on an N x N grid: edge conductances are the means of their
    two unknowns' conductivities, the boundary conducts with 1."""

    def __init__(self, n, device):
        rowptr, col, _ = W.poisson_csr(n, np.int32)
        self.n = n
        self.pattern = K.sla_csr_create_from_csr(torch.from_numpy(rowptr).to(device),
                                                 torch.from_numpy(col).to(device))
        count = torch.from_numpy(rowptr).long().diff()
        self.row = torch.repeat_interleave(torch.arange(n * n), count).to(device)
        self.col = torch.from_numpy(col).long().to(device)
        self.off = (self.row != self.col)
        self.outer = (4 - (count - 1)).double().to(device)  # edges to the boundary

    def matrix(self, log_conductivity):
        c = log_conductivity.reshape(-1).double().exp()
        edge = torch.where(self.off, 0.5 * (c[self.row] + c[self.col]), 0.0)
        diag = torch.zeros_like(c).index_add(0, self.row, edge) + self.outer
        return K.SparseTensor(self.pattern, torch.where(self.off, -edge, diag[self.row]))

    def solve(self, log_conductivity, b, tol=1e-10):
        return K.solve(self.matrix(log_conductivity), b, tol=tol, maxit=10 * self.n * self.n)


def problem(n, device, seed=0):
    """Features [n, n, 5], the hidden log conductivity and the right-hand side."""
    gen = torch.Generator().manual_seed(seed)
    y, x = torch.meshgrid(torch.linspace(0, 1, n), torch.linspace(0, 1, n), indexing="ij")
    blob = torch.exp(-((x - 0.35) ** 2 + (y - 0.6) ** 2) / 0.04)
    wave = torch.sin(7 * x) * torch.cos(5 * y)
    noise = 0.1 * torch.randn(n, n, generator=gen)
    features = torch.stack([x, y, blob, wave, noise], -1).to(device)
    hidden = (1.2 * blob - 0.6 * wave).to(device)
    return features, hidden, torch.ones(n * n, dtype=torch.float64, device=device)


def train(n=32, steps=40, dtype=torch.float32, lr=5e-3, seed=0, mixer="delta", optimizer="adam"):
    """(the loss of every step, network, features)"""
    device = torch.device("cuda")
    torch.manual_seed(seed)
    features, hidden, b = problem(n, device, seed)
    kind = {"delta": Network, "scan": ScanNetwork}[mixer]
    grid, net = Diffusion(n, device), kind(dtype=dtype).to(device)
    with torch.no_grad():
        wanted = grid.solve(hidden, b)
    opt = {"adam": torch.optim.Adam, "orthogonal": Orthogonalised}[optimizer](net.parameters(),
                                                                              lr=lr)
    losses = []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        x = grid.solve(net(features), b)
        loss = (x - wanted).square().sum() / wanted.square().sum()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses, net, features


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--grid", type=int, default=32)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--mixer", choices=("delta", "scan"), default="delta")
    ap.add_argument("--optimizer", choices=("adam", "orthogonal"), default="adam")
    args = ap.parse_args()
    losses, net, features = train(args.grid, args.steps, mixer=args.mixer,
                                  optimizer=args.optimizer)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  relative squared error {losses[i]:.3e}")
    with torch.no_grad():
        whole = net(features)
    one = net.step_by_step(features)
    print(f"last step {losses[-1]:.3e}; token by token differs by "
          f"{float((one - whole).abs().max()):.1e}")


if __name__ == "__main__":
    main()
