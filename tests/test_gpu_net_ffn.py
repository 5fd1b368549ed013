"""The gated feed-forward unit on the GPU against its 64-bit form.

Bounds, element by element, from sums of absolute terms (u = half a step of
the tensors' type, U32 of fp32; slopes of the activations are at most 1.13):
  a, b   off by (inner + 2) U32 (|x| |W|^T)
  h      u |h| + 1.13 da_err |b| + |f(a)| db_err + 16 U32 (|a| + 1)(|b| + 1)
  da, db rounded to the type once: u relative, beside what a and b carry
  dx, dw that, summed over absolute terms, plus (terms) U32, plus u of the result
Where the slope of relu jumps (a near 0) it may fall on either side: such
elements widen the bound by the whole term."""
import pytest
import torch

import net_refs as R

pytestmark = pytest.mark.gpu

CASES = [  # rows, inner, outer
    (1, 1, 1), (1, 64, 64), (4, 96, 40), (3, 7, 130), (33, 100, 65), (128, 64, 128),
    (130, 33, 67), (65, 515, 140), (257, 128, 256), (300, 72, 200), (16, 256, 128), (17, 64, 96),
    (0, 32, 48), (512, 256, 384),
]


def inputs(rows, inner, outer, dtype, seed=0):
    g = R.gen(seed + rows * 7 + inner)
    x = torch.randn(rows, inner, generator=g)
    wg = torch.randn(outer, inner, generator=g) / inner ** 0.5
    wu = torch.randn(outer, inner, generator=g) / inner ** 0.5
    dh = torch.randn(rows, outer, generator=g)
    return [t.to(dtype) for t in (x, wg, wu, dh)]


def bounds(x, wg, wu, dh, act, u):
    """Wanted outputs and how far each may be off."""
    inner, outer, rows = x.shape[1], wg.shape[0], x.shape[0]
    a = (x @ wg.t()).requires_grad_()
    b = x @ wu.t()
    ea = (inner + 2) * R.U32 * (x.abs() @ wg.abs().t())
    eb = (inner + 2) * R.U32 * (x.abs() @ wu.abs().t())
    f = R.activation(a, act)
    (df,) = torch.autograd.grad(f.sum(), a)
    a, f = a.detach(), f.detach()
    near = 16 * R.U32 * (a.abs() + 1)
    h = f * b
    eh = u * h.abs() + 1.13 * ea * b.abs() + f.abs() * eb + near * (b.abs() + 1)
    da, db = dh * b * df, dh * f
    jump = ((a.abs() <= ea).double() if act == "relu" else ea)  # the slope's error (f'' <= 1)
    ea2 = u * da.abs() + dh.abs() * (eb * 1.13 + b.abs() * (jump + near))
    eb2 = u * db.abs() + dh.abs() * (1.13 * ea + near)
    dx = da @ wg + db @ wu
    edx = u * dx.abs() + ea2 @ wg.abs() + eb2 @ wu.abs() + \
        (2 * outer + 2) * R.U32 * (da.abs() @ wg.abs() + db.abs() @ wu.abs())
    dwg, dwu = da.t() @ x, db.t() @ x
    edg = u * dwg.abs() + ea2.t() @ x.abs() + (rows + 2) * R.U32 * (da.abs().t() @ x.abs())
    edu = u * dwu.abs() + eb2.t() @ x.abs() + (rows + 2) * R.U32 * (db.abs().t() @ x.abs())
    return {"h": (h, eh), "dx": (dx, edx), "dwg": (dwg, edg), "dwu": (dwu, edu)}


def close(got, want, tol, what):
    d = (got.detach().double().cpu() - want).abs()
    # 1 + 2^-6: second-order terms of the bounds above
    bad = d > tol * (1 + 2 ** -6) + 1e-300
    assert not bad.any(), (what, d[bad].max().item(), tol[bad].max().item(), int(bad.sum()))


@pytest.mark.parametrize("rows, inner, outer", CASES)
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gated_ffn_and_gradients(rows, inner, outer, kind, act):
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    x, wg, wu, dh = inputs(rows, inner, outer, dtype)
    leaves = [t.cuda().requires_grad_() for t in (x, wg, wu)]
    h = K.gated_ffn(*leaves, act)
    dx, dwg, dwu = torch.autograd.grad(h, leaves, dh.cuda())
    assert h.dtype == dx.dtype == dwg.dtype == dtype and h.shape == (rows, outer)
    if rows == 0:
        assert not dwg.any() and not dwu.any()
        return
    # fp16's smallest steps: absolute 2^-25
    tiny = 2.0 ** -25 * 4 if kind == "fp16" else 0.0
    want = bounds(*(t.double() for t in (x, wg, wu, dh)), act, R.half_step(dtype))
    for name, got in (("h", h), ("dx", dx), ("dwg", dwg), ("dwu", dwu)):
        ref, tol = want[name]
        close(got, ref, tol + tiny * (1 + max(rows, outer)), name)
    with torch.no_grad():
        assert torch.equal(K.gated_ffn(*leaves, act), h.detach())


def test_large_arguments_of_the_activations():
    import krylov_solvers_adjoint_amd as K
    x = torch.tensor([[100.0], [-100.0], [1e4], [-1e4], [float("inf")], [float("nan")], [0.0]])
    one = torch.ones(1, 1)
    for act in ("silu", "gelu", "relu"):
        leaf = x.cuda().requires_grad_()
        h = K.gated_ffn(leaf, one.cuda(), one.cuda(), act)
        (dx,) = torch.autograd.grad(h, leaf, torch.ones_like(h))
        want = R.gated_ffn(x.double(), one.double(), one.double(), act)
        fine = x[:, 0].isfinite()
        assert R.rel(h.cpu()[fine], want[fine]) < 1e-6
        assert dx.cpu()[fine].isfinite().all()
        assert h.cpu()[5].isnan().all() and h.cpu()[4].isinf().all()


def test_views_and_leading_axes():
    import krylov_solvers_adjoint_amd as K
    g = R.gen(3)
    base = torch.randn(2, 19, 210, generator=g).to(torch.bfloat16).cuda()
    wg, wu = (torch.randn(70, 101, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    for view in (base[..., 5:106], base[:, ::3, 5:106], base[0, :, 1:102]):
        leaves = [view.detach().requires_grad_(), wg.detach().requires_grad_(),
                  wu.detach().requires_grad_()]
        h = K.gated_ffn(*leaves)
        dh = torch.ones(1, device="cuda", dtype=h.dtype).expand_as(h)   # strides of zero
        got = torch.autograd.grad(h, leaves, dh)
        whole = [t.detach().contiguous().requires_grad_() for t in leaves]
        hw = K.gated_ffn(*whole)
        want = torch.autograd.grad(hw, whole, torch.ones_like(hw))
        assert h.shape == (*view.shape[:-1], 70) and torch.equal(h, hw)
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_only_some_gradients_and_refusals():
    import krylov_solvers_adjoint_amd as K
    x, wg, wu, dh = (t.cuda() for t in inputs(20, 40, 50, torch.float32))
    full = [t.clone().requires_grad_() for t in (x, wg, wu)]
    want = torch.autograd.grad(K.gated_ffn(*full), full, dh)
    for keep in (0, 1, 2):
        some = [t.clone().requires_grad_(i == keep) for i, t in enumerate((x, wg, wu))]
        (got,) = torch.autograd.grad(K.gated_ffn(*some), some[keep], dh)
        assert torch.equal(got, want[keep])
    with pytest.raises(ValueError):
        K.gated_ffn(x, wg, wu, "tanh")
    with pytest.raises(TypeError):
        K.gated_ffn(x, wg.half(), wu)
    with pytest.raises(ValueError):
        K.gated_ffn(x, wg[:, :39], wu[:, :39])
    with pytest.raises(ValueError):
        K.gated_ffn(x, wg, wu[:49])
    with pytest.raises(TypeError):
        K.gated_ffn(x.double(), wg.double(), wu.double())


def test_against_differences():
    import krylov_solvers_adjoint_amd as K
    x, wg, wu, dh = (t.cuda() for t in inputs(200, 96, 150, torch.float32))
    for act in ("silu", "gelu"):
        leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
        grads = torch.autograd.grad(K.gated_ffn(*leaves, act), leaves, dh)
        step = [torch.randn(t.shape, generator=R.gen(9)).cuda() * 1e-2 * t.std() for t in (x, wg, wu)]
        lo, hi = (K.gated_ffn(*[t + s * d for t, d in zip((x, wg, wu), step)], act).double()
                  for s in (-1, 1))
        num = ((hi - lo) * dh.double()).sum().item() / 2
        ana = sum((p.double() * d.double()).sum().item() for p, d in zip(grads, step))
        # h^2 = 1e-4 of third derivatives of order one
        assert abs(num - ana) < 1e-3 * ((hi - lo).norm() * dh.double().norm()).item() / 2


def test_graph_replays_and_other_streams():
    import krylov_solvers_adjoint_amd as K
    x, wg, wu, dh = (t.cuda() for t in inputs(300, 128, 256, torch.bfloat16))

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, wg, wu)]
        h = K.gated_ffn(*leaves)
        return (h.detach(), *torch.autograd.grad(h, leaves, dh))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(torch.randn(300, 128, generator=R.gen(20 + k)))
        graph.replay()
        torch.cuda.synchronize()
        again = step()
        torch.cuda.synchronize()
        for p, q in zip(out, again):
            assert torch.equal(p, q)
