"""The network operators where their first form was wrong or lost digits."""
import math

import pytest
import torch

import net_refs as R
import test_gpu_net_delta as D

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Gates that reset the state
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("reset", [-1e4, -1e16, -1e20, torch.finfo(torch.float32).min, -math.inf])
@pytest.mark.parametrize("places", [[0], [20], [63], [64, 65], [3, 4, 40, 127, 149]])
def test_gates_that_reset_the_state(reset, places):
    """Against the recurrence, gradients too (the bound of every other gate),
    and token by token.  Gates of -1e16 and below took the later ones out of a
    running sum; -inf made NaN of a chunk."""
    import krylov_solvers_adjoint_amd as K
    ins, do, ds = D.inputs(1, 150, 1, 2, 32, 48, torch.float32)
    ins[3][:, places] = reset
    o, state = D.compare(ins, do, ds)
    leaves = [t.cuda().requires_grad_() for t in ins]
    out = K.gated_delta_rule(*leaves[:5], initial_state=leaves[5], output_final_state=True)
    (dg,) = torch.autograd.grad(out, leaves[3], (do.cuda(), ds.cuda()))
    assert not dg[:, places].any()
    q, k, v, g, beta, kept = (t.cuda() for t in ins)
    for t in range(150):
        one = K.gated_delta_step(q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t], kept)
        assert R.rel(one, o[:, t]) <= 4 * D.TOL
    assert R.rel(kept, state) <= 2 * D.TOL


def test_a_gate_that_is_no_number_shows():
    import krylov_solvers_adjoint_amd as K
    ins, _, _ = D.inputs(1, 70, 1, 1, 16, 16, torch.float32)
    ins[3][0, 30] = math.nan
    o, s = K.gated_delta_rule(*(t.cuda() for t in ins[:5]), initial_state=ins[5].cuda(),
                              output_final_state=True)
    assert o[0, 30:].isnan().all() and s.isnan().all()


# ---------------------------------------------------------------------------
# Forward-mode derivatives
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused(grad):
    """They were dropped: a result without a tangent stands for a zero one."""
    import krylov_solvers_adjoint_amd as K
    import torch.autograd.forward_ad as fw
    x = torch.randn(1, 5, 2, 16, device="cuda")
    w = torch.randn(24, 16, device="cuda")
    g = -torch.rand(1, 5, 2, device="cuda")
    s = torch.zeros(1, 2, 16, 16, device="cuda")
    with fw.dual_level(), torch.set_grad_enabled(grad):
        d = fw.make_dual(x, torch.ones_like(x))
        dg = fw.make_dual(g, torch.ones_like(g))
        for call in (lambda: K.layer_norm(d), lambda: K.gated_ffn(d, w, w),
                     lambda: K.gated_ffn(x, w, fw.make_dual(w, w)),
                     lambda: K.gated_delta_rule(d, x, x, g, g),
                     lambda: K.gated_delta_rule(x, x, x, dg, g)):
            with pytest.raises(NotImplementedError):
                call()
        with pytest.raises(ValueError):
            K.gated_delta_step(x[:, 0], x[:, 0], x[:, 0], dg[:, 0], g[:, 0], s)
        assert not s.any()
        # nothing that carries a tangent: as ever
        assert torch.equal(K.layer_norm(x), K.layer_norm(x.clone()))
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda t: K.layer_norm(t), (x,), (x,))
