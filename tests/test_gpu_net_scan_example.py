"""The example's lighter network (gated scans, projections with epilogues) and its
optimiser (orthogonalised updates), as they are used together: its gradient is the
loss's, token by token it gives what it gives at once, a training step runs through
the adjoint solve, also replayed from a graph, and moves every weight as it should."""
import os
import sys

import pytest
import torch

import net_refs as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_runs_and_tokens_agree(dtype):
    import coefficient_network as C
    losses, net, features = C.train(n=20, steps=4, dtype=dtype, mixer="scan",
                                    optimizer="orthogonal")
    assert all(torch.isfinite(torch.tensor(losses))) and len(losses) == 4
    with torch.no_grad():
        whole = net(features)
    one = net.step_by_step(features)
    # a rounding of every tensor on the way more or less: a few half steps of the type
    tol = 64 * torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 1e-4
    assert (one - whole).abs().max() <= tol * whole.abs().max().clamp_min(1)


def test_gradient_against_differences():
    import coefficient_network as C
    device = torch.device("cuda")
    torch.manual_seed(3)
    features, hidden, b = C.problem(12, device)
    grid, net = C.Diffusion(12, device), C.ScanNetwork().to(device)
    wanted = grid.solve(hidden, b).detach()

    def loss():
        return (grid.solve(net(features), b, tol=1e-12) - wanted).square().sum()
    grads = torch.autograd.grad(loss(), list(net.parameters()))
    step = [torch.randn_like(p.detach()) * 1e-3 * p.detach().abs().mean().clamp_min(0.1)
            for p in net.parameters()]
    ana = sum(float((g.double() * s.double()).sum()) for g, s in zip(grads, step))
    ends = []
    with torch.no_grad():
        for sign in (1, -2):
            for p, s in zip(net.parameters(), step):
                p.add_(s, alpha=sign)
            ends.append(float(loss()))
    num = (ends[0] - ends[1]) / 2
    # fp32 network: rounding 1e-6 of the loss over a change of 1e-3 of it, and the step's curvature
    assert abs(num - ana) <= 2e-2 * max(abs(num), abs(ana)), (num, ana)


def test_network_against_elementary_operations():
    """The block as a whole, values and gradients, against torch in 64 bits."""
    import coefficient_network as C
    torch.manual_seed(5)
    net = C.ScanNetwork().cuda()
    features = torch.randn(7, 33, 5, generator=R.gen(1)).cuda()
    leaf = features.clone().requires_grad_()
    out = net(leaf)
    grads = torch.autograd.grad(out.square().sum(), [leaf, *net.parameters()])
    p = {n: t.detach().double().requires_grad_() for n, t in net.named_parameters()}
    x = features.double().requires_grad_()

    def norm(h, i):
        return R.layer_norm(h, p[f"norms.{i}.0"], p[f"norms.{i}.1"], 1e-5)
    h = R.activation(x @ p["enter"].t() + p["enter_bias"], "gelu")
    n = norm(h, 0)
    a = torch.exp(-torch.nn.functional.softplus(n @ p["gate"].t() + p["gate_bias"]))
    v = n @ p["value"].t()
    state, rows = torch.zeros_like(v[:, 0]), []
    for t in range(v.shape[1]):
        state = a[:, t] * state + v[:, t]
        rows.append(state)
    h = h + torch.stack(rows, 1) @ p["mix"].t()
    f = R.gated_ffn(norm(h, 1), p["w_gate"], p["w_up"], "silu")
    h = h + f @ p["w_down"].t()
    ref = (norm(h, 2) @ p["head"].t() + p["head_bias"])[..., 0]
    want = torch.autograd.grad(ref.square().sum(), [x, *p.values()])
    # some twenty fp32 operators in a row, sums of up to 231 tokens
    assert R.rel(out, ref) <= 1e-5
    for got, w, name in zip(grads, want, ["x", *p]):
        assert R.rel(got, w) <= 1e-4, name


def test_a_step_of_the_optimiser():
    import coefficient_network as C
    torch.manual_seed(1)
    w = torch.randn(48, 130, device="cuda").requires_grad_()
    tall = torch.randn(100, 20, device="cuda").requires_grad_()
    b = torch.randn(30, device="cuda").requires_grad_()
    before = [t.detach().clone() for t in (w, tall, b)]
    opt = C.Orthogonalised([w, tall, b], lr=0.1)
    for t in (w, tall, b):
        t.grad = torch.randn(t.shape, generator=R.gen(7)).cuda()
    opt.step()
    for t, old, size in ((w, before[0], 1.0), (tall, before[1], 5 ** 0.5)):
        s = torch.linalg.svdvals((old - t.detach()).double().cpu() / (0.1 * size))
        assert s.min() > 0.6 and s.max() < 1.3   # all directions alike
    # Adam's first step is lr in the gradient's direction
    assert torch.allclose(before[2] - b.detach(), 0.1 * b.grad.sign(), rtol=1e-4, atol=1e-5)


def test_the_block_replayed_from_a_graph():
    import coefficient_network as C
    torch.manual_seed(2)
    net = C.ScanNetwork(dtype=torch.bfloat16).cuda()
    features = torch.randn(4, 200, 5, generator=R.gen(2)).cuda()
    params = list(net.parameters())

    def step():
        # leaves of its own: a graph of the eager run's leaves must not live on
        own = {n: p.detach().requires_grad_() for n, p in net.named_parameters()}
        out = torch.func.functional_call(net, own, (features,))
        return (out.detach(), *torch.autograd.grad(out.square().sum(), list(own.values())))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    assert len(out) == 1 + len(params)
    for k in range(3):
        features.copy_(torch.randn(4, 200, 5, generator=R.gen(30 + k)))
        graph.replay()
        torch.cuda.synchronize()
        again = step()
        torch.cuda.synchronize()
        for p, q in zip(out, again):
            assert torch.equal(p, q)
