"""The example that trains a network of these operators through the solver's
adjoint: its loss falls, its gradient is the loss's, and token by token it
gives what it gives at once."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_through_the_adjoint(dtype):
    import coefficient_network as C
    losses, net, features = C.train(n=20, steps=30, dtype=dtype)
    assert losses[-1] < 0.3 * losses[0], losses
    with torch.no_grad():
        whole = net(features)
    one = net.step_by_step(features)
    # one rounding of q, k, v and o more or less: a few half steps of the type
    tol = 64 * torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 1e-4
    assert (one - whole).abs().max() <= tol * whole.abs().max().clamp_min(1)


def test_gradient_against_differences():
    import coefficient_network as C
    device = torch.device("cuda")
    torch.manual_seed(3)
    features, hidden, b = C.problem(12, device)
    grid, net = C.Diffusion(12, device), C.Network().to(device)
    wanted = grid.solve(hidden, b).detach()

    def loss():
        return (grid.solve(net(features), b, tol=1e-12) - wanted).square().sum()
    grads = torch.autograd.grad(loss(), list(net.parameters()))
    step = [torch.randn_like(p.detach()) * 1e-3 * p.detach().abs().mean() for p in net.parameters()]
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
