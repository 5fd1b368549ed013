"""What the network operators refuse, on the CPU: bad arguments never reach a
kernel.  The C entries are called with made-up addresses that they must
reject before any of them is used."""
import ctypes

import pytest
import torch

import krylov_solvers_adjoint_amd as K
from krylov_solvers_adjoint_amd import network as net

lib = K._lib
P = 256  # an address that is never followed


def last():
    return lib.sla_last_error().decode()


def test_layer_norm_refusals():
    n = K._I64()
    ok = dict(x=P, ld=8, rows=4, cols=8, t=0, w=P, b=P, wt=0, eps=1e-5, y=P)

    def call(**kw):
        a = {**ok, **kw}
        return lib.sla_layer_norm(a["x"], a["ld"], a["rows"], a["cols"], a["t"], a["w"], a["b"],
                                  a["wt"], a["eps"], a["y"], None, None)
    for kw in (dict(x=None), dict(y=None), dict(ld=7), dict(rows=-1), dict(rows=1 << 31),
               dict(cols=0), dict(t=3), dict(t=-1), dict(wt=1), dict(wt=2), dict(eps=-1.0),
               dict(eps=float("nan"))):
        assert call(**kw) == K.ERR_ARG, kw
        assert last().startswith("sla_layer_norm"), kw
    assert call(rows=0, x=None, y=None) == K.OK  # nothing to do
    assert lib.sla_layer_norm_work(4, 8, 0, None) == K.ERR_ARG
    assert lib.sla_layer_norm_work(4, 8, 0, ctypes.byref(n)) == K.OK and n.value > 0
    # dw wanted, but the workspace is missing or short
    for work, size in ((None, n.value), (P, n.value - 1)):
        assert lib.sla_layer_norm_grad(P, 8, P, 8, 4, 8, 0, P, 0, P, P, P, P, work, size,
                                       None) == K.ERR_ARG
        assert "workspace" in last()
    assert lib.sla_layer_norm_grad(None, 8, P, 8, 4, 8, 0, P, 0, P, P, P, P, P, n.value,
                                   None) == K.ERR_ARG
    assert lib.sla_layer_norm_grad(P, 7, P, 8, 4, 8, 0, P, 0, P, P, P, P, P, n.value,
                                   None) == K.ERR_ARG


def test_gated_ffn_refusals():
    def call(x=P, ld=8, wg=P, wu=P, rows=4, inner=8, outer=16, t=0, act=0, h=P):
        return lib.sla_gated_ffn(x, ld, wg, wu, rows, inner, outer, t, act, h, None)
    for kw in (dict(x=None), dict(wg=None), dict(wu=None), dict(h=None), dict(ld=7),
               dict(rows=-1), dict(inner=0), dict(outer=0), dict(t=9), dict(act=3), dict(act=-1),
               dict(rows=1 << 40), dict(outer=1 << 40)):
        assert call(**kw) == K.ERR_ARG, kw
        assert last().startswith("sla_gated_ffn"), kw
    assert call(rows=0, x=None, h=None) == K.OK
    n = K._I64()
    assert lib.sla_gated_ffn_work(4, 8, 16, 2, ctypes.byref(n)) == K.OK
    # lddh, dh, the workspace, one weight's gradient without the other's
    good = [P, 16, P, 8, P, P, 4, 8, 16, 2, 0, P, P, P, P, n.value, None]
    for at, bad in ((0, None), (1, 15), (2, None), (3, 7), (12, None), (14, None),
                    (15, n.value - 1)):
        args = list(good)
        args[at] = bad
        assert lib.sla_gated_ffn_grad(*args) == K.ERR_ARG, at


def dims(**kw):
    d = dict(sequences=2, tokens=8, key_heads=2, value_heads=4, key_dim=16, value_dim=24,
             scale=1.0, type=0, packed=0)
    d.update(kw)
    return net._DeltaDims(*[d[n] for n, _ in net._DeltaDims._fields_])


def test_delta_refusals():
    n, m = K._I64(), K._I64()
    for kw in (dict(type=5), dict(sequences=-1), dict(tokens=-1), dict(tokens=9),
               dict(sequences=0), dict(key_heads=0), dict(value_heads=3), dict(value_heads=0),
               dict(key_dim=0), dict(key_dim=129), dict(value_dim=0), dict(value_dim=4097),
               dict(tokens=1 << 31, packed=1)):
        assert lib.sla_delta_rule_work(ctypes.byref(dims(**kw)), ctypes.byref(n),
                                       None) == K.ERR_ARG, kw
    assert lib.sla_delta_rule_work(None, None, None) == K.ERR_ARG
    d = dims()
    assert lib.sla_delta_rule_work(ctypes.byref(d), ctypes.byref(n), ctypes.byref(m)) == K.OK
    good = [ctypes.byref(d), P, 32, P, 32, P, 96, P, P, None, None, P, P, P, n.value, None]
    for at, bad in ((1, None), (2, 31), (3, None), (4, 31), (5, None), (6, 95), (7, None),
                    (8, None), (11, None), (13, None), (14, n.value - 1)):
        args = list(good)
        args[at] = bad
        assert lib.sla_delta_rule(*args) == K.ERR_ARG, at
    packed = dims(packed=1)
    args = list(good)
    args[0] = ctypes.byref(packed)
    args[14] = 1 << 40
    assert lib.sla_delta_rule(*args) == K.ERR_ARG and "offsets" in last()
    good = [ctypes.byref(d), P, 32, P, 32, P, 96, P, P, P, n.value, P, 96, None, P, P, P, P, P, P,
            P, m.value, None]
    for at, bad in ((1, None), (9, None), (10, n.value - 1), (11, None), (12, 95), (20, None),
                    (21, m.value - 1)):
        args = list(good)
        args[at] = bad
        assert lib.sla_delta_rule_grad(*args) == K.ERR_ARG, at
    one = dims(tokens=2)
    good = [ctypes.byref(one), P, 32, P, 32, P, 96, P, P, P, P, None]
    for at, bad in ((0, ctypes.byref(dims())), (0, ctypes.byref(dims(tokens=2, packed=1))),
                    (1, None), (9, None), (10, None), (6, 95)):
        args = list(good)
        args[at] = bad
        assert lib.sla_delta_step(*args) == K.ERR_ARG, at
    # no sequences: nothing to do
    assert lib.sla_delta_rule(ctypes.byref(dims(sequences=0, tokens=0)), *([None] * 1), 32, None,
                              32, None, 96, None, None, None, None, None, None, None, 0,
                              None) == K.OK


def test_cpu_tensors_and_wrong_kinds_are_refused():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.layer_norm(x)
    with pytest.raises(TypeError):
        K.layer_norm([1.0])
    with pytest.raises(ValueError, match="GPU tensor"):
        K.gated_ffn(x, x, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.gated_delta_rule(x, x, x, x, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        K.gated_delta_step(x, x, x, x, x, x)


@pytest.mark.parametrize("make, tail, ld", [
    (lambda: torch.zeros(6, 8), 1, 8),
    (lambda: torch.zeros(6, 20)[:, 4:12], 1, 20),           # part of a wider row
    (lambda: torch.zeros(2, 3, 20)[..., :8], 1, 20),
    (lambda: torch.zeros(1, 3, 40)[..., 8:24].unflatten(-1, (2, 8)), 2, 40),
    (lambda: torch.zeros(1, 8)[:, :3], 1, 8),
])
def test_views_with_even_rows_are_taken_as_they_are(make, tail, ld):
    t = make()
    u, got = net._rows(t, tail)
    assert u.data_ptr() == t.data_ptr() and (got == ld or t.shape[0] == 1)


@pytest.mark.parametrize("make, tail", [
    (lambda: torch.zeros(8, 6).t(), 1),                     # rows not contiguous
    (lambda: torch.zeros(6, 1).expand(6, 8), 1),            # broadcast columns
    (lambda: torch.zeros(1, 8).expand(6, 8), 1),            # broadcast rows
    (lambda: torch.zeros(3, 2, 8).transpose(0, 1), 1),      # rows in another order
    (lambda: torch.zeros(4, 3, 2, 8).transpose(1, 2), 2),   # heads before tokens
    (lambda: torch.zeros(4, 6, 8)[:, :4], 1),               # gaps between batches
])
def test_other_views_are_copied(make, tail):
    t = make()
    u, ld = net._rows(t, tail)
    assert u.is_contiguous() and u.shape == t.shape and torch.equal(u, t)
    width = 1
    for n in t.shape[t.dim() - tail:]:
        width *= n
    assert ld == width


def test_tangents_go_to_the_autograd_nodes_and_are_refused_there():
    """A dual tensor does not require grad: called directly, a kernel would drop
    its tangent in silence."""
    import torch.autograd.forward_ad as fw
    x = torch.randn(3, 4)
    assert not net._wants(x, None)
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        assert not net._wants(x, None)
        assert net._wants(x, None, d)
        with torch.no_grad():
            assert net._wants(d)
    y = x.clone()
    with fw.dual_level(), pytest.MonkeyPatch.context() as m:
        m.setattr(net, "sla_layer_norm", lambda *a, **k: (y, y))
        m.setattr(net, "sla_gated_ffn", lambda *a, **k: y)
        m.setattr(net, "sla_delta_rule", lambda *a, **k: (y, y, y))
        d = fw.make_dual(x, torch.ones_like(x))
        for call in (lambda: net._LayerNorm.apply(d, x, x, 1e-5),
                     lambda: net._GatedFFN.apply(x, d, x, 0),
                     lambda: net._DeltaRule.apply(x, x, x, d, x, None, None, 1, 1.0, True)):
            with pytest.raises(NotImplementedError):
                call()


def test_another_stream_gets_the_copies_and_the_memory_too(monkeypatch):
    """With stream= everything of an sla_* call happens on that stream.  Memory
    of the current stream's pool would go back to it on return, while the
    kernels on the other stream still use it."""
    import contextlib
    import types
    inside, seen = [None], []
    other = types.SimpleNamespace(cuda_stream=77)

    @contextlib.contextmanager
    def on(stream):
        inside[0] = stream.cuda_stream
        yield
        inside[0] = None
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda raw, device=None: types.SimpleNamespace(cuda_stream=raw))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: inside[0] or 11,
                        raising=False)
    empty, empty_like = torch.empty, torch.empty_like

    def allocate(make):
        def call(*a, **k):
            seen.append(("memory", inside[0]))
            return make(*a, **k)
        return call
    monkeypatch.setattr(torch, "empty", allocate(empty))
    monkeypatch.setattr(torch, "empty_like", allocate(empty_like))
    rows = net._rows

    def copied(t, tail):
        seen.append(("copy", inside[0]))
        return rows(t, tail)
    monkeypatch.setattr(net, "_rows", copied)

    def kernel(*args):
        seen.append(("kernel", args[-1]))
        return 0
    names = ("sla_layer_norm", "sla_layer_norm_grad", "sla_gated_ffn", "sla_gated_ffn_grad",
             "sla_delta_rule", "sla_delta_rule_grad", "sla_delta_step")
    monkeypatch.setattr(net, "_lib", types.SimpleNamespace(**{n: kernel for n in names}))
    monkeypatch.setattr(net, "_work_bytes", lambda *a: 64)
    monkeypatch.setattr(net, "_delta_dims", lambda *a: (dims(), None, 64, 64))
    x, w, stats = torch.zeros(8, 4).t(), torch.zeros(16, 8), torch.zeros(4, 2)
    q = torch.zeros(2, 4, 2, 16)
    v, gate = torch.zeros(2, 4, 4, 24), torch.zeros(2, 4, 4)
    s = torch.zeros(2, 4, 16, 24)
    calls = {
        "sla_layer_norm": (x, None, None, 1e-5, True),
        "sla_layer_norm_grad": (x, x, None, stats, True, True, True, None),
        "sla_gated_ffn": (x, w, w, 0),
        "sla_gated_ffn_grad": (torch.zeros(4, 16), x, w, w, 0, True, True),
        "sla_delta_rule": (q, q, v, gate, gate, None, None, 2, 1.0, True),
        "sla_delta_rule_grad": (q, q, v, gate, gate, s, v, None, 2, 1.0, False, True),
        "sla_delta_step": (q[:, 0], q[:, 0], v[:, 0], gate[:, 0], gate[:, 0], s, 1.0),
    }
    for name in names:
        f, args = getattr(net, name), calls[name]
        for how in (lambda: f(*args, other), lambda: f(*args, stream=other),
                    lambda: f(*args, stream=77)):
            seen.clear()
            how()
            assert {what for what, _ in seen} == {"memory", "copy", "kernel"}
            assert all(stream == 77 for _, stream in seen), (name, seen)
        seen.clear()
        f(*args)
        assert all(stream in (None, 11) for _, stream in seen), (name, seen)


def test_a_step_counts_as_a_change_of_its_state(monkeypatch):
    """The kernel writes through a pointer; autograd learns of it by the version."""
    import types
    monkeypatch.setattr(net, "_lib", types.SimpleNamespace(sla_delta_step=lambda *a: 0))
    monkeypatch.setattr(net, "_delta_dims", lambda *a: (dims(), None, 64, 64))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    q, gate = torch.zeros(2, 1, 4), torch.zeros(2, 1)
    leaf = torch.randn(2, 1, 4, 4, requires_grad=True)
    state = leaf.clone()
    loss = state.square().sum()
    net.sla_delta_step(q, q, q, gate, gate, state.detach(), 1.0)
    assert state._version == 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        net.sla_delta_step(q, q, q, gate, gate, torch.zeros(2, 1, 4, 4), 1.0)


def test_walks_of_2_to_the_32_threads_are_refused():
    """The runtime would start only a part of them (sequences without tokens:
    with tokens what they keep would not fit the card)."""
    d = dims(sequences=1 << 23, tokens=0, key_heads=1, value_heads=1)
    assert lib.sla_delta_rule(ctypes.byref(d), None, 32, None, 32, None, 96, None, None, None, P,
                              None, P, P, 1 << 50, None) == K.ERR_ARG
    assert "too many" in last()
    assert lib.sla_delta_rule_grad(ctypes.byref(d), None, 32, None, 32, None, 96, None, None, P,
                                   1 << 50, None, 96, P, None, None, None, None, None, P, P,
                                   1 << 50, None) == K.ERR_ARG
    assert "too many" in last()


def test_rows_of_the_feed_forward_unit():
    """As many as layer norm's: a row an unknown, the framework's grids have 1.7e8."""
    n = K._I64()
    for rows in (1 << 22, 169_000_000, (1 << 31) - 1):
        assert lib.sla_gated_ffn_work(rows, 8, 16, 2, ctypes.byref(n)) == K.OK, rows
        assert n.value >= 2 * rows * 16 * 2
    assert lib.sla_gated_ffn_work(1 << 31, 8, 16, 2, ctypes.byref(n)) == K.ERR_ARG
    # no launch of 2^32 threads
    assert lib.sla_gated_ffn(P, 8, P, P, (1 << 31) - 1, 8, 4096, 2, 0, P, None) == K.ERR_ARG
    assert "too large" in last()


def test_assembly_names_the_registers_it_writes():
    """m0 holds the LDS address of a direct load: the compiler uses it too."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(K.__file__), "csrc")
    for name in sorted(os.listdir(csrc)):
        if name.endswith((".hip", ".h")):
            with open(os.path.join(csrc, name)) as f:
                text = f.read()
            for block in re.findall(r"asm volatile\((.*?)\);", text, re.S):
                if re.search(r"s_mov_b32 m0", block):
                    assert '"m0"' in block.rsplit(":", 1)[1], (name, block)
