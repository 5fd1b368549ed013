"""The projection, the gated scan and the orthogonalised update where their first
form was wrong, lost digits or was not looked at."""
import math

import pytest
import torch

import net_refs as R
import test_gpu_net_linear as L

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


# ---------------------------------------------------------------------------
# The bias's gradient
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows, inner, outer", [(64, 32, 32), (65, 64, 64), (300, 9, 64),
                                                (130, 61, 50), (100, 33, 17), (257, 64, 32),
                                                (4096, 64, 64)])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_a_wide_bias_gradient_of_narrow_projections_is_summed_unrounded(rows, inner, outer, kind,
                                                                        act):
    """A bias in fp32 has a gradient whose terms were never rounded to 16 bits: the linear tests'
    bound of db without u |dz|."""
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    x, w, b, r, dy = L.inputs(rows, inner, outer, dtype, torch.float32)
    leaves = [t.cuda().requires_grad_() for t in (x, w, b)]
    db = torch.autograd.grad(K.linear(*leaves, act), leaves, dy.cuda())[2]
    x, w, b, dy = (t.double() for t in (x, w, b, dy))
    z = x @ w.t() + b
    ez = (inner + 3) * R.U32 * (x.abs() @ w.abs().t() + b.abs())
    z.requires_grad_()
    (slope,) = torch.autograd.grad(R.activation(z, act).sum(), z)
    z = z.detach()
    near = 16 * R.U32 * (z.abs() + 1) + (1.2e-5 * (z.abs() + 1) if act == "gelu" else 0)
    jump = (z.abs() <= ez).double() if act == "relu" else ez
    dz = dy * slope
    tol = R.U32 * dz.sum(0).abs() + (dy.abs() * (jump + near)).sum(0) \
        + (rows + 2) * R.U32 * dz.abs().sum(0)
    if act == "relu":   # the slopes are exact: fp32's sums are all that is rounded
        tol = R.U32 * dz.sum(0).abs() + (dy.abs() * jump).sum(0) \
            + (rows + 2) * R.U32 * dz.abs().sum(0)
    L.close(db, dz.sum(0), tol, "db")
