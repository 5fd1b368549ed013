"""The projection, the gated scan and the orthogonalised update where their first
form was wrong, lost digits or was not looked at."""
import math

import pytest
import torch

import net_refs as R

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Gates that grow
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind, gkind", [("fp32", "fp32"), ("bf16", "fp32"), ("fp16", "fp32"),
                                         ("bf16", "bf16"), ("fp16", "fp16")])
def test_a_gate_whose_exp_leaves_the_range_gives_infinity(kind, gkind):
    """exp(g) above 2^128 is infinite, not NaN, whatever the last bits of g; below it the decay has
    its digits, and NaN stays NaN."""
    import krylov_solvers_adjoint_amd as K
    dtype, gtype = R.TYPES[kind], R.TYPES[gkind]
    g = torch.cat([torch.linspace(80, 88.7, 301), torch.linspace(88.75, 201, 3001),
                   torch.tensor([250.0, 1e4, math.inf])]).to(gtype)
    n = g.numel()
    zero = torch.zeros(1, n, dtype=dtype).cuda()
    want = g.double().exp()
    inside = want < torch.finfo(torch.float32).max
    assert 200 < int(inside.sum()) < n - 2000
    for start in (1.0, -0.5):
        state = torch.full((1, n), start).cuda()
        K.gated_scan_step(zero, g[None].cuda(), state)
        h, last = K.gated_scan(zero[None], g[None, None].cuda(), torch.full((1, n), start).cuda(),
                               True)
        for got in (state[0].cpu(), last[0].cpu()):
            assert torch.equal(got[~inside], torch.full_like(got[~inside], math.inf * start))
            # 2 ulp of exp, and one rounding; 16-bit gates leave |g| 2^-23.5
            tol = 6 * R.U32 if gkind == "fp32" else 6 * R.U32 + 90 * 2.0 ** -23.5
            assert ((got[inside].double() - start * want[inside]).abs()
                    <= tol * want[inside]).all()
    state = torch.ones(1, n).cuda()
    nan = torch.full((1, n), math.nan, dtype=gtype).cuda()
    K.gated_scan_step(zero, nan, state)
    assert state.isnan().all()
