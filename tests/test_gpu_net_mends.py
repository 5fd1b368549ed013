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
