"""The network operators at sizes that reach their large tiles, split sums and
long walks, against 64-bit forms; the bounds are those of the small tests."""
import pytest
import torch

import net_refs as R
import test_gpu_net_delta as D
import test_gpu_net_ffn as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows, inner, outer", [
    (4120, 1032, 2088),   # whole 16-byte units: the largest tiles, cut at every edge
    (4096, 256, 2048),    # ... and nothing cut
    (2000, 517, 1403),    # odd widths: tiles staged by way of registers
    (300, 2040, 520),     # long sums, few tiles
])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_gated_ffn(rows, inner, outer, kind):
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    x, wg, wu, dh = (t.cuda() for t in F.inputs(rows, inner, outer, dtype))
    leaves = [t.requires_grad_() for t in (x, wg, wu)]
    h = K.gated_ffn(*leaves, "silu")
    dx, dwg, dwu = torch.autograd.grad(h, leaves, dh)
    want = F.bounds(*(t.detach().double() for t in (x, wg, wu, dh)), "silu", R.half_step(dtype))
    tiny = 2.0 ** -25 * 4 if kind == "fp16" else 0.0
    for name, got in (("h", h), ("dx", dx), ("dwg", dwg), ("dwu", dwu)):
        ref, tol = want[name]
        d = (got.detach().double() - ref).abs()
        bad = d > (tol + tiny * (1 + max(rows, outer))) * (1 + 2 ** -6)
        assert not bad.any(), (name, d[bad].max().item(), int(bad.sum()))
    again = torch.autograd.grad(K.gated_ffn(*leaves, "silu"), leaves, dh)
    for p, q in zip((dx, dwg, dwu), again):
        assert torch.equal(p, q)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hk, hv, dk, dv", [(2, 4, 128, 96), (1, 1, 64, 200), (2, 2, 100, 40)])
def test_long_sequences(kind, hk, hv, dk, dv):
    D.compare(*D.inputs(1, 600, hk, hv, dk, dv, R.TYPES[kind], decay=0.1))


def test_values_of_many_sizes_keep_their_precision():
    """States and values from 1e-20 to 1e20 in one sequence: parts of eight bits
    have the range of fp32, so the bound holds column by column."""
    import krylov_solvers_adjoint_amd as K
    ins, _, _ = D.inputs(1, 130, 1, 1, 64, 64, torch.float32)
    q, k, v, g, beta, s0 = ins
    size = 10.0 ** torch.linspace(-20, 20, 64)
    v, s0 = v * size, s0 * size
    o, s = K.gated_delta_rule(*(t.cuda() for t in (q, k, v, g, beta)), initial_state=s0.cuda(),
                              output_final_state=True)
    o64, s64 = R.delta_rule(*(t.double() for t in (q, k, v, g, beta, s0)), 1 / 8)
    for c in range(0, 64, 7):
        assert R.rel(o[..., c], o64[..., c]) <= D.TOL
        assert R.rel(s[..., c], s64[..., c]) <= D.TOL


@pytest.mark.parametrize("rows, cols", [(200000, 64), (3000, 1024), (20000, 97)])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_layer_norm(rows, cols, kind):
    import krylov_solvers_adjoint_amd as K
    import test_gpu_net_norm as N
    x, w, b, dy = (t.cuda() for t in N.inputs(rows, cols, R.TYPES[kind], R.TYPES[kind]))
    leaves = [t.requires_grad_() for t in (x, w, b)]
    got = (y := K.layer_norm(*leaves), *torch.autograd.grad(y, leaves, dy))
    ref = [t.detach().double().requires_grad_() for t in leaves]
    y64 = R.layer_norm(*ref, 1e-5)
    want = (y64, *torch.autograd.grad(y64, ref, dy.double()))
    u = R.half_step(R.TYPES[kind])
    for p, q in zip(got, want):
        assert R.rel(p, q) <= u + 100 * R.U32
