"""The network operators where their first form was wrong or lost digits."""
import math

import pytest
import torch

import net_refs as R
import test_gpu_net_delta as D
import test_gpu_net_ffn as F

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


# ---------------------------------------------------------------------------
# Another stream
# ---------------------------------------------------------------------------
def test_another_stream_gives_the_same_bits_and_owns_what_it_returns():
    import krylov_solvers_adjoint_amd as K
    from krylov_solvers_adjoint_amd import network as net
    side = torch.cuda.Stream()

    def pool(t):
        for seg in torch.cuda.memory_snapshot():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                return seg["stream"]
    base = torch.randn(200, 96, generator=R.gen(1)).cuda()
    x, w = base[:, 3:67], torch.randn(128, 64, generator=R.gen(2)).cuda()
    xt = torch.randn(64, 200, generator=R.gen(3)).cuda().t()      # copied
    dh = torch.randn(200, 128, generator=R.gen(4)).cuda()
    ins, do, ds = D.inputs(2, 100, 1, 2, 32, 48, torch.float32)
    q, k, v, g, beta, s0 = (t.cuda() for t in ins)
    do, ds = do.cuda(), ds.cuda()

    def all_of(stream):
        y, stats = net.sla_layer_norm(xt, None, None, 1e-5, True, stream=stream)
        out = [y, *net.sla_layer_norm_grad(x, xt, None, stats, stream=stream)]
        out.append(net.sla_gated_ffn(xt, w, w, 0, stream=stream))
        out += net.sla_gated_ffn_grad(dh, x, w, w, 0, stream=stream)
        o, s, kept = net.sla_delta_rule(q, k, v, g, beta, None, s0, 2, 0.2, stream=stream)
        out += [o, s, *net.sla_delta_rule_grad(q, k, v, g, beta, kept, do, ds, 2, 0.2, False,
                                               stream=stream)]
        kept = s0.clone()
        torch.cuda.synchronize()
        out.append(net.sla_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(),
                                      beta[:, 0].contiguous(), kept, 0.2, stream=stream))
        torch.cuda.synchronize()
        return [*out, kept]
    want = all_of(None)
    for stream in (side, side.cuda_stream, 0):
        torch.cuda.synchronize()
        got = all_of(stream)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        owner = 0 if stream == 0 else side.cuda_stream
        assert all(pool(t) == owner for t in got[:-1])
    torch.cuda.synchronize()


def test_the_operators_on_a_side_stream_give_the_bits_of_the_default_one():
    import krylov_solvers_adjoint_amd as K
    x = torch.randn(300, 64, generator=R.gen(1)).cuda()
    w = torch.randn(96, 64, generator=R.gen(2)).cuda()
    ins, do, ds = D.inputs(1, 150, 1, 2, 32, 48, torch.bfloat16)
    dev = [t.cuda() for t in ins]
    do, ds = do.cuda(), ds.cuda()

    def all_of():
        a, b, c = (t.clone().requires_grad_() for t in (x, w, w))
        n = K.layer_norm(a, b[0], c[0])
        h = K.gated_ffn(n, b, c)
        out = [n.detach(), h.detach(), *torch.autograd.grad(h.sum(), (a, b, c))]
        leaves = [t.clone().requires_grad_() for t in dev]
        o, s = K.gated_delta_rule(*leaves[:5], initial_state=leaves[5], output_final_state=True)
        return [*out, o.detach(), s.detach(), *torch.autograd.grad((o, s), leaves, (do, ds))]
    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# A state that a graph has saved
# ---------------------------------------------------------------------------
def test_a_step_on_a_saved_state_is_noticed():
    import krylov_solvers_adjoint_amd as K
    ins, _, _ = D.inputs(1, 20, 1, 2, 16, 24, torch.float32)
    leaves = [t.cuda().requires_grad_() for t in ins]
    _, state = K.gated_delta_rule(*leaves[:5], initial_state=leaves[5], output_final_state=True)
    loss = state.square().sum()
    with torch.no_grad():
        K.gated_delta_step(*(t[:, 0] for t in leaves[:5]), state.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


# ---------------------------------------------------------------------------
# Activations
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 80])
def test_relu_of_minus_infinity_is_zero(kind, rows):
    """a overflows to -inf where the definition has 0 and a slope of 0."""
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    x = torch.full((rows, 1), 3e38).to(dtype)
    wg, wu = torch.tensor([[-3e38]]).to(dtype), torch.tensor([[1e-38]]).to(dtype)
    leaves = [t.cuda().requires_grad_() for t in (x, wg, wu)]
    h = K.gated_ffn(*leaves, "relu")
    assert not h.any() and h.isfinite().all()
    for t in torch.autograd.grad(h, leaves, torch.ones_like(h)):
        assert not t.any() and t.isfinite().all()
    # what is no number stays that, in h and in the gradients
    leaves[0] = torch.full_like(leaves[0], math.nan).requires_grad_()
    h = K.gated_ffn(*leaves, "relu")
    assert h.isnan().all()
    for t in torch.autograd.grad(h, leaves, torch.ones_like(h)):
        assert t.isnan().all()


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("few", [True, False])
def test_gelu_keeps_its_relative_precision_in_the_tail(kind, few):
    """f(a) b for single values of a (exact in the type), b = 2^15 so that fp16
    holds f down to 2^-29: the output's rounding (half a step) and 2^-15 for
    exp, its argument's rounding and the fit, all relative."""
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    a = torch.linspace(-12, 3, 4001).to(dtype)
    x = torch.stack([a, torch.ones_like(a)], 1)
    wg, wu = (torch.tensor([w]).to(dtype) for w in ([1.0, 0.0], [0.0, 2.0 ** 15]))
    parts = x.cuda().split(50) if few else [x.cuda()]
    h = torch.cat([K.gated_ffn(p, wg.cuda(), wu.cuda(), "gelu") for p in parts])[:, 0]
    want = R.activation(a.double(), "gelu") * 2.0 ** 15
    tol = (R.half_step(dtype) + 2.0 ** -15) * want.abs()
    tol += 2.0 ** -25 if kind == "fp16" else 2.0 ** -126     # the type's smallest steps
    held = want.abs() <= torch.finfo(dtype).max
    bad = ~((h.cpu().double() - want).abs() <= tol) & held
    assert not bad.any(), (a[bad], ((h.cpu().double() - want).abs() / want.abs())[bad].max())


@pytest.mark.parametrize("few", [True, False])
def test_gelu_keeps_its_relative_precision_in_fp32(few):
    """f(a) by itself (b = 1): erfc's argument is rounded once, which its tail
    multiplies by a^2; 32 roundings for erfc, the products and the output."""
    import krylov_solvers_adjoint_amd as K
    a = torch.linspace(-12, 6, 4001)
    x = torch.stack([a, torch.ones_like(a)], 1)
    wg, wu = torch.tensor([[1.0, 0.0]]), torch.tensor([[0.0, 1.0]])
    parts = x.cuda().split(50) if few else [x.cuda()]
    h = torch.cat([K.gated_ffn(p, wg.cuda(), wu.cuda(), "gelu") for p in parts])[:, 0]
    a = a.double()
    want = R.activation(a, "gelu")
    bad = ~((h.cpu().double() - want).abs() <= (2 * a * a + 32) * R.U32 * want.abs())
    assert not bad.any(), (a[bad], ((h.cpu().double() - want).abs() / want.abs())[bad].max())


# ---------------------------------------------------------------------------
# fp16's range between the products of the feed-forward unit's gradient
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows, inner, outer", [(40, 64, 96), (300, 64, 96), (300, 65, 97),
                                                (4096, 256, 2048)])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("size", ["tiny", "small", "one", "large"])
def test_fp16_gradients_hold_for_every_size_of_dh(rows, inner, outer, act, size):
    """dx and dW are ordinary fp16 numbers, the products between them are not:
    below 2^-24 (tiny: dh = 5 of fp16's smallest steps and less, large x and W)
    or beyond 65504.  The bounds are the operator's own, beside 2^-38 of the
    largest |da| or |db| that the norms allow (fp16's smallest half step at the
    scale they are held) and half of fp16's smallest step in the output."""
    import krylov_solvers_adjoint_amd as K
    g = R.gen(rows + outer)
    x = torch.rand(rows, inner, generator=g) - 0.25
    wg = torch.randn(outer, inner, generator=g) / inner ** 0.5
    wu = torch.randn(outer, inner, generator=g) / inner ** 0.5
    dh = torch.rand(rows, outer, generator=g) - 0.25
    sx, sg, su, sd = {"tiny": (1.0, 512.0, 0.5, 4e-7), "small": (64.0, 0.01, 0.01, 3e-5),
                      "one": (1.0, 1.0, 1.0, 1.0), "large": (0.01, 0.01, 3e3, 4e3)}[size]
    x, wg, wu, dh = ((t * s).half().cuda() for t, s in ((x, sx), (wg, sg), (wu, su), (dh, sd)))
    leaves = [t.requires_grad_() for t in (x, wg, wu)]
    got = torch.autograd.grad(K.gated_ffn(*leaves, act), leaves, dh)
    x, wg, wu, dh = (t.detach().double() for t in (x, wg, wu, dh))
    want = F.bounds(x, wg, wu, dh, act, R.half_step(torch.float16))
    most = 1.13 * dh.abs().max() * x.norm(dim=1).max() * max(wg.norm(dim=1).max(),
                                                              wu.norm(dim=1).max())
    tiny = 2.0 ** -38 * most
    more = {"dx": tiny * (wg.abs().sum(0) + wu.abs().sum(0)),
            "dwg": tiny * x.abs().sum(0), "dwu": tiny * x.abs().sum(0)}
    for name, t in zip(("dx", "dwg", "dwu"), got):
        ref, tol = want[name]
        tol = (tol + more[name]) * (1 + 2 ** -6) + 2.0 ** -25
        t = t.double()
        # of the largest case some results themselves lie beyond fp16: infinities
        near = ((t - ref).abs() <= tol) | ((t == ref.sign() * math.inf) & (ref.abs() + tol >= 65520))
        assert near.all(), (name, int((~near).sum()), t[~near][:4], ref[~near][:4])
        assert size == "large" or t.isfinite().all()


def test_fp16_gradients_beside_values_that_are_not_finite():
    """A row of them leaves the other rows' dx as they are without it."""
    import krylov_solvers_adjoint_amd as K
    x, wg, wu, dh = (t.cuda() for t in F.inputs(100, 64, 96, torch.float16))

    def dx_of(x, dh):
        leaf = x.clone().requires_grad_()
        return torch.autograd.grad(K.gated_ffn(leaf, wg, wu), leaf, dh)[0]
    want = dx_of(x, dh)
    x2, dh2 = x.clone(), dh.clone()
    x2[3, 5], x2[70, 1], dh2[9, 9], dh2[60, 2] = math.inf, math.nan, math.inf, math.nan
    got = dx_of(x2, dh2)
    good = torch.ones(100, dtype=torch.bool)
    good[[3, 70, 9, 60]] = False
    # the scale may be another power of two: the same up to fp16's smallest steps
    assert R.rel(got[good], want[good]) <= 2.0 ** -11
    assert not got[~good].isfinite().all(1).any()
    zero = dx_of(x, torch.zeros_like(dh))
    assert not zero.any() and zero.isfinite().all()


# ---------------------------------------------------------------------------
# Results that cancel
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("heads", [1, 2])
def test_outputs_behind_erasing_tokens(kind, heads):
    """Eight tokens erase eight rows of a state of 1e3 (beta = 1, keys of one
    element, no decay) and write values of 1; every token asks for the mean of
    those rows, and grad_o asks for one column.  What is left of 1e3 keeps
    fp32's digits: 40 roundings of the terms before they cancel, then the
    output's.  (Factors of two 8-bit parts, cut off at 2^-16, left 0.015.)"""
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    g = R.gen(8)
    q, k = torch.zeros(1, 9, 1, 64), torch.zeros(1, 9, 1, 64)
    k[0, range(8), 0, range(8)] = 1
    q[..., :8] = 0.25
    v = torch.randn(1, 9, heads, 64, generator=g)
    beta, gate = torch.ones(1, 9, heads), torch.zeros(1, 9, heads)
    s0 = 1e3 * torch.randn(1, heads, 64, 64, generator=g)
    do = torch.zeros(1, 9, heads, 64)
    for t in range(9):
        do[0, t, :, 7 * t + 3] = 1
    ins = [t.to(dtype) for t in (q, k, v)] + [gate, beta, s0]
    leaves = [t.cuda().requires_grad_() for t in ins]
    o, _ = K.gated_delta_rule(*leaves[:5], initial_state=leaves[5])
    dq, dk = torch.autograd.grad(o, leaves[:2], do.to(dtype).cuda())
    ref = [t.double().requires_grad_() for t in ins]
    o64, _ = R.delta_rule(*ref, 1 / 8)
    rq, rk = torch.autograd.grad(o64, ref[:2], do.double())
    u = R.half_step(dtype)
    size = s0.double().abs() + 4                                   # of the terms
    tol = u * o64.detach().abs() + 40 * R.U32 / 8 * 0.25 * size[0, :, :8].sum(1)
    assert ((o.detach().cpu().double() - o64.detach()).abs() <= tol).all()
    each = torch.stack([size[0, :, :, 7 * t + 3].sum(0) for t in range(9)])[None, :, None]
    near = (dq.cpu().double() - rq).abs() <= u * rq.abs() + 40 * R.U32 / 8 * each
    assert near.all(), ((dq.cpu().double() - rq).abs() / each / R.U32).max()
    assert R.rel(dk, rk) <= u + D.TOL


# ---------------------------------------------------------------------------
# Launches of 2^32 threads
# ---------------------------------------------------------------------------
def test_weight_gradients_of_more_than_2_to_the_26_columns():
    """All but 18 columns were never written: one row, so db is dy itself and dw
    is dy times the normalised row, one rounding each."""
    import krylov_solvers_adjoint_amd as K
    n = (1 << 26) + 5
    x = torch.rand(1, n, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    w = torch.ones(n, device="cuda", requires_grad=True)
    b = torch.zeros(n, device="cuda", requires_grad=True)
    y = K.layer_norm(x, w, b)
    dw, db = torch.autograd.grad(y, (w, b), x)
    assert torch.equal(db, x[0])
    assert ((dw - x[0] * y[0]).abs() <= 4 * R.U32 * dw.abs()).all()


def test_steps_of_more_than_2_to_the_24_states():
    """Half of the outputs and states were left as they were."""
    import krylov_solvers_adjoint_amd as K
    n = (1 << 24) - 1
    one, two = torch.ones(n, 1, 1, device="cuda"), torch.ones(n, 2, 1, device="cuda")
    v = torch.arange(2 * n, device="cuda").remainder(1 << 20).float().view(n, 2, 1)
    s = torch.zeros(n, 2, 1, 1, device="cuda")
    o = K.gated_delta_step(one, one, v, torch.zeros(n, 2, device="cuda"), two[..., 0], s)
    assert torch.equal(o, v) and torch.equal(s[..., 0], v)


# ---------------------------------------------------------------------------
# Layer norm: rows with an outlier, far means, long rows
# ---------------------------------------------------------------------------
def norm_rows(cols, kind):
    """Rows of N(0, 1) with one outlier (first, last), far means, and both."""
    g = R.gen(cols)
    top = {"fp32": 1e8, "bf16": 1e8, "fp16": 6e4}[kind]
    far = {"fp32": 1e6, "bf16": 1e2, "fp16": 1e3}[kind]
    x = torch.randn(9, cols, generator=g)
    x[0, 0], x[1, 0], x[2, 0], x[3, -1] = 1e4, top / 50, -top, top
    x[4] += far
    x[5] += far
    x[5, 0] = 0
    x[6] += far
    x[6, 0] = top
    x[7] = x[7, 0]
    return x.to(R.TYPES[kind])


@pytest.mark.parametrize("cols", [2, 8, 40, 257, 1000, 2000, 4100, 8192, 8200, 20001])
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
def test_layer_norm_keeps_every_element_s_digits(cols, kind):
    """Element by element, each at its own size: an element's deviation d carries
    one rounding and the mean's, 40 (sums of 32 values a lane and the team's)
    of the mean |d|; the statistic 1 / sqrt(var + eps) 60 relative ones.  The
    gradient's deviation has the mean rounded once more, at its distance from
    zero or the first element, whichever is nearer.  With differences to the
    first element, its rounding was on every other one."""
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    x = norm_rows(cols, kind)
    g = R.gen(1)
    w = (1 + 0.1 * torch.randn(cols, generator=g)).to(dtype)
    dy = torch.randn(x.shape, generator=g).to(dtype)
    xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = K.layer_norm(xd, wd)
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.cuda())
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    y64 = R.layer_norm(x64, w64, None, 1e-5)
    rx, rw = torch.autograd.grad(y64, (x64, w64), dy.double())
    x64, w64, dy = x64.detach(), w64.detach(), dy.double()
    U, u = R.U32, R.half_step(dtype)
    mean = x64.mean(1, keepdim=True)
    d = x64 - mean
    rstd = 1 / (d.square().mean(1, keepdim=True) + 1e-5).sqrt()
    n = d * rstd
    base = 80 * d.abs().mean(1, keepdim=True)
    en = U * (rstd * (2 * d.abs() + base) + 60 * n.abs())
    tol = u * y64.detach().abs() + (en + 4 * U * n.abs()) * w64.abs()
    near = (y.detach().cpu().double() - y64.detach()).abs() <= tol
    assert near.all(), (near.logical_not().nonzero()[:5], (y.cpu().double() - y64)[~near][:5])
    x0 = x64[:, :1]
    zero = mean.abs() < (mean - x0).abs()
    start, left = torch.where(zero, 0, x0), torch.where(zero, mean, mean - x0)
    eb = en + U * rstd * ((x64 - start).abs() + 2 * left.abs())
    t = dy * w64
    s1, s2 = t.abs().mean(1, keepdim=True), (t * n).abs().mean(1, keepdim=True)
    e2 = (t.abs() * eb).mean(1, keepdim=True) + 60 * U * s2
    tol = u * rx.abs() + rstd * (60 * U * (t.abs() + s1 + n.abs() * s2)
                                 + eb * (t * n).mean(1, keepdim=True).abs() + n.abs() * e2)
    near = (dx.cpu().double() - rx).abs() <= tol * (1 + 2 ** -6) + (2.0 ** -25 if kind == "fp16" else 0)
    assert near.all(), (near.logical_not().nonzero()[:5], (dx.cpu().double() - rx)[~near][:5])
    tol = u * rw.abs() + (dy.abs() * eb).sum(0) + 60 * U * (dy * n).abs().sum(0)
    assert ((dw.cpu().double() - rw).abs() <= tol * (1 + 2 ** -6)).all()
    assert not y[7].any()      # a constant row


def test_layer_norm_of_a_long_row():
    """2e7 columns: 78125 values a thread, summed in fp64; what is left is the
    rounding of a few elementwise steps."""
    import krylov_solvers_adjoint_amd as K
    x = 1 + torch.rand(1, 20_000_000, generator=torch.Generator("cuda").manual_seed(2),
                       device="cuda")
    dy = torch.randn(x.shape, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    leaf = x.clone().requires_grad_()
    y = K.layer_norm(leaf)
    (dx,) = torch.autograd.grad(y, leaf, dy)
    x64 = x.double().requires_grad_()
    y64 = R.layer_norm(x64, None, None, 1e-5)
    (rx,) = torch.autograd.grad(y64, x64, dy.double())
    assert R.rel(y, y64) <= 8 * R.U32 and R.rel(dx, rx) <= 16 * R.U32


# ---------------------------------------------------------------------------
# The feed-forward unit: a row an unknown
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows, inner, outer, kind", [
    ((1 << 22) + 77, 8, 16, "bf16"), ((1 << 22) + 77, 5, 3, "fp32"), (16_000_000, 16, 8, "fp16")])
def test_more_than_2_to_the_22_rows(rows, inner, outer, kind):
    """They were refused.  h and dx element by element; dW is a sum of `rows`
    terms in fp32, whose roundings add up like a random walk."""
    import krylov_solvers_adjoint_amd as K
    dtype = R.TYPES[kind]
    gen = torch.Generator("cuda").manual_seed(rows)
    x, wg, wu, dh = (torch.randn(s, generator=gen, device="cuda") * c
                     for s, c in (((rows, inner), 1), ((outer, inner), inner ** -0.5),
                                  ((outer, inner), inner ** -0.5), ((rows, outer), 0.01)))
    x, wg, wu, dh = (t.to(dtype) for t in (x, wg, wu, dh))
    leaves = [t.requires_grad_() for t in (x, wg, wu)]
    h = K.gated_ffn(*leaves)
    got = dict(zip(("dx", "dwg", "dwu"), torch.autograd.grad(h, leaves, dh)), h=h)
    want = F.bounds(*(t.detach().double() for t in (x, wg, wu, dh)), "silu", R.half_step(dtype))
    for name in ("h", "dx"):
        ref, tol = want[name]
        tiny = 2.0 ** -25 if kind == "fp16" else 0
        assert ((got[name].detach().double() - ref).abs() <= tol * (1 + 2 ** -6) + tiny).all(), name
    for name in ("dwg", "dwu"):
        assert R.rel(got[name], want[name][0]) <= 2 * R.half_step(dtype) + rows ** 0.5 * R.U32


# ---------------------------------------------------------------------------
# Offsets
# ---------------------------------------------------------------------------
def test_offsets_that_are_no_whole_numbers_are_refused():
    """A list of them was cut off: 1.7 became 1."""
    import numpy as np
    import krylov_solvers_adjoint_amd as K
    ins, _, _ = D.inputs(1, 6, 1, 1, 8, 8, torch.float32)
    q, k, v, g, beta, _ = (t.cuda() for t in ins)
    for bad in ([0, 1.7, 6], [0.0, 6.0], np.array([0.5, 6.0]), [True, True]):
        with pytest.raises(TypeError):
            K.gated_delta_rule(q, k, v, g, beta, cu_seqlens=bad)
    with pytest.raises(ValueError):
        K.gated_delta_rule(q, k, v, g, beta, cu_seqlens=[])
    want = K.gated_delta_rule(q, k, v, g, beta, cu_seqlens=[0, 2, 6])[0]
    for good in ((0, 2, 6), np.array([0, 2, 6]), np.array([0, 2, 6], dtype=np.int32),
                 torch.tensor([0, 2, 6]), torch.tensor([0, 2, 6]).cuda()):
        assert torch.equal(K.gated_delta_rule(q, k, v, g, beta, cu_seqlens=good)[0], want)


# ---------------------------------------------------------------------------
# What a comparison with ">" lets pass
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
def test_no_output_is_other_than_finite(kind):
    """The element by element bounds of layer norm and the feed-forward unit ask
    whether a difference is larger than its bound, which no NaN is."""
    import krylov_solvers_adjoint_amd as K
    import test_gpu_net_norm as N
    dtype = R.TYPES[kind]
    for rows, cols in N.CASES:
        x, w, b, dy = (t.cuda() for t in N.inputs(rows, cols, dtype, dtype))
        leaves = [t.requires_grad_() for t in (x, w, b)]
        y = K.layer_norm(*leaves)
        for t in (y, *torch.autograd.grad(y, leaves, dy)):
            assert t.isfinite().all(), (rows, cols)
    for rows, inner, outer in F.CASES + [(1030, 264, 520)]:
        for act in ("silu", "gelu", "relu"):
            x, wg, wu, dh = (t.cuda() for t in F.inputs(rows, inner, outer, dtype))
            leaves = [t.requires_grad_() for t in (x, wg, wu)]
            h = K.gated_ffn(*leaves, act)
            for t in (h, *torch.autograd.grad(h, leaves, dh)):
                assert t.isfinite().all(), (rows, inner, outer, act)


def test_the_fp16_gradient_in_a_graph():
    """Its scale is found anew in every replay, from that replay's inputs."""
    import krylov_solvers_adjoint_amd as K
    x, wg, wu, dh = (t.cuda() for t in F.inputs(300, 128, 256, torch.float16))

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
    first = F.inputs(300, 128, 256, torch.float16)[3].cuda()
    for size in (2.0 ** -14, 1.0, 2.0 ** 8, 2.0 ** -8):
        dh.copy_(first * size)
        graph.replay()
        torch.cuda.synchronize()
        again = step()
        torch.cuda.synchronize()
        for p, q in zip(out, again):
            assert torch.equal(p, q) and p.isfinite().all()


# ---------------------------------------------------------------------------
# The gates' gradient behind strong decays
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [-2.0, -5.0, -10.0, -20.0, -60.0])
def test_gradient_of_strong_gates(gate, kind):
    """dg is as small as exp(g) then, and has the digits of every other gradient:
    the operator's bound holds for it by itself.  (Sums of everything from a
    token on, in which what does not cross the token cancels, had left 5e-3 at
    -10 and noise of 1e9 times dg at -60.)"""
    ins, do, ds = D.inputs(1, 150, 1, 2, 32, 48, R.TYPES[kind])
    ins[3].fill_(gate)
    D.compare(ins, do, ds)


@pytest.mark.parametrize("shape", [(1, 300, 2, 2, 64, 64), (2, 130, 1, 3, 100, 40)])
def test_gradient_of_strong_gates_among_weak_ones(shape):
    """By the size of the gate: the strong ones' gradients are not lost beside
    the weak ones'."""
    import krylov_solvers_adjoint_amd as K
    batch, tokens, hk, hv, dk, dv = shape
    ins, do, ds = D.inputs(batch, tokens, hk, hv, dk, dv, torch.float32)
    which = torch.randint(0, 4, ins[3].shape, generator=R.gen(3))
    sizes = torch.tensor([-0.01, -1.0, -12.0, -40.0])
    ins[3].copy_(sizes[which])
    leaves = [t.cuda().requires_grad_() for t in ins]
    out = K.gated_delta_rule(*leaves[:5], initial_state=leaves[5], output_final_state=True)
    (dg,) = torch.autograd.grad(out, leaves[3], (do.cuda(), ds.cuda()))
    ref = [t.double().requires_grad_() for t in ins]
    out = R.delta_rule(*ref, dk ** -0.5)
    (rg,) = torch.autograd.grad(out, ref[3], (do.double(), ds.double()))
    for n in range(4):
        assert R.rel(dg.cpu()[which == n], rg[which == n]) <= D.TOL, sizes[n]
