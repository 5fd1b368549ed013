"""What the projection, the gated scan and the orthogonalised update refuse, on
the CPU: bad arguments never reach a kernel.  The C entries are called with
made-up addresses that they must reject before any of them is used."""
import contextlib
import ctypes
import types

import pytest
import torch

import krylov_solvers_adjoint_amd as K
from krylov_solvers_adjoint_amd import network as net

lib = K._lib
P = 256  # an address that is never followed


def last():
    return lib.sla_last_error().decode()


def refused(entry, good, bad):
    for at, value in bad:
        args = list(good)
        args[at] = value
        assert getattr(lib, entry)(*args) == K.ERR_ARG, (entry, at, value)
        assert last().startswith(entry), (entry, at, value, last())


def test_linear_refusals():
    f, n = K._I64(), K._I64()
    assert lib.sla_linear_work(4, 8, 16, 2, 0, ctypes.byref(f), ctypes.byref(n)) == K.OK
    assert lib.sla_linear_work(4, 8, 16, 2, 3, None, None) == K.OK
    refused("sla_linear_work", [4, 8, 16, 2, 0, None, None],
            [(0, -1), (0, 1 << 31), (1, 0), (1, 1 << 22), (2, 0), (2, 1 << 22), (3, 3), (3, -1),
             (4, 4), (4, -1)])
    # x, ldx, weight, bias, btype, residual, ldr, rows, inner, outer, type, act, y, work, bytes
    good = [P, 8, P, P, 2, P, 16, 4, 8, 16, 2, 0, P, P, 1 << 30, None]
    refused("sla_linear", good, [(0, None), (1, 7), (2, None), (4, 1), (4, 3), (6, 15), (7, -1),
                                 (8, 0), (9, 0), (10, 5), (11, 4), (12, None)])
    none = list(good)
    none[0] = none[12] = None
    none[7] = 0
    assert lib.sla_linear(*none) == K.OK  # no rows: nothing to do
    # sums of a split product
    assert lib.sla_linear_work(100, 200000, 64, 2, 3, ctypes.byref(f), None) == K.OK and f.value
    split = [P, 200000, P, None, 2, None, 0, 100, 200000, 64, 2, 3, P, P, f.value, None]
    refused("sla_linear", split, [(13, None), (14, f.value - 1)])
    good = [P, 16, P, 8, P, P, 2, 4, 8, 16, 2, 0, P, P, P, P, n.value, None]
    refused("sla_linear_grad", good, [(0, None), (1, 15), (2, None), (3, 7), (4, None), (6, 1),
                                      (7, -1), (10, 9), (11, 7), (15, None), (16, n.value - 1)])


def dims(**kw):
    d = dict(sequences=2, tokens=8, channels=24, type=2, gate_type=0, packed=0)
    d.update(kw)
    return net._ScanDims(*[d[n] for n, _ in net._ScanDims._fields_])


def test_scan_refusals():
    n, m = K._I64(), K._I64()
    refused("sla_gated_scan_work", [ctypes.byref(dims()), None, None],
            [(0, ctypes.byref(dims(**kw))) for kw in (
                dict(type=3), dict(type=-1), dict(gate_type=1), dict(sequences=-1),
                dict(tokens=-1), dict(tokens=9), dict(sequences=0), dict(channels=0),
                dict(channels=1 << 31), dict(tokens=1 << 31, packed=1),
                dict(sequences=0, packed=1), dict(sequences=1, tokens=1 << 39, channels=1 << 30))]
            + [(0, None)])
    d = dims()
    assert lib.sla_gated_scan_work(ctypes.byref(d), ctypes.byref(n), ctypes.byref(m)) == K.OK
    good = [ctypes.byref(d), P, 24, P, 24, None, None, P, P, P, n.value, P, m.value, None]
    refused("sla_gated_scan", good, [(0, None), (1, None), (2, 23), (3, None), (4, 23), (7, None),
                                     (10, n.value - 1)])
    packed = dims(packed=1)
    assert lib.sla_gated_scan_work(ctypes.byref(packed), ctypes.byref(n), ctypes.byref(m)) == K.OK
    good = [ctypes.byref(packed), P, 24, P, 24, P, None, P, P, P, n.value, P, m.value, None]
    refused("sla_gated_scan", good, [(5, None), (10, n.value - 1), (11, None), (12, m.value - 1)])
    good = [ctypes.byref(packed), P, 24, P, 24, P, n.value, P, 24, None, P, P, P, P, m.value, None]
    refused("sla_gated_scan_grad", good,
            [(0, None), (1, None), (2, 23), (3, None), (4, 23), (5, None), (6, n.value - 1),
             (7, None), (8, 23), (13, None), (14, m.value - 1)])
    one = dims(tokens=2)
    good = [ctypes.byref(one), P, 24, P, 24, P, P, None]
    refused("sla_gated_scan_step", good,
            [(0, ctypes.byref(dims())), (0, ctypes.byref(dims(tokens=2, packed=1))), (0, None),
             (1, None), (2, 23), (3, None), (4, 23), (5, None), (6, None)])
    # no sequences: nothing to do
    none = ctypes.byref(dims(sequences=0, tokens=0))
    assert lib.sla_gated_scan(none, None, 24, None, 24, None, None, None, None, None, 0, None, 0,
                              None) == K.OK
    assert lib.sla_gated_scan_step(none, None, 24, None, 24, None, None, None) == K.OK


def test_orthogonalise_refusals():
    n = K._I64()
    refused("sla_orthogonalise_work", [2, 8, 9, 0, ctypes.byref(n)],
            [(0, -1), (0, 65536), (1, 0), (1, 65537), (2, 0), (2, 65537), (3, 3), (4, None)])
    assert lib.sla_orthogonalise_work(2, 8, 9, 0, ctypes.byref(n)) == K.OK and n.value == 0
    assert lib.sla_orthogonalise_work(2, 200, 300, 0, ctypes.byref(n)) == K.OK and n.value > 0
    c = (ctypes.c_double * 3)(1.5, -0.5, 0.0)
    nan = (ctypes.c_double * 3)(1.5, float("nan"), 0.0)
    big = (ctypes.c_double * 3)(1.5, -65.0, 0.0)
    good = [P, 300, 2, 200, 300, 0, 1, c, 1e-7, P, P, n.value, None]
    refused("sla_orthogonalise", good,
            [(0, None), (1, 299), (2, -1), (3, 0), (4, 0), (5, 4), (6, -1), (6, 65), (7, None),
             (7, nan), (7, big), (8, -1.0), (8, float("nan")), (9, None), (10, None),
             (11, n.value - 1)])
    good[2] = 0
    assert lib.sla_orthogonalise(*good) == K.OK


def test_cpu_tensors_and_wrong_kinds_are_refused():
    x = torch.zeros(4, 8)
    for call in (lambda: K.linear(x, x), lambda: K.gated_scan(x[None], x[None]),
                 lambda: K.gated_scan_step(x, x, x), lambda: K.orthogonalise(x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: K.linear([1.0], x), lambda: K.gated_scan(None, x),
                 lambda: K.orthogonalise([[1.0]])):
        with pytest.raises(TypeError):
            call()


def test_tangents_are_refused_by_the_autograd_nodes():
    import torch.autograd.forward_ad as fw
    x = torch.randn(3, 4)
    with fw.dual_level(), pytest.MonkeyPatch.context() as m:
        m.setattr(net, "sla_linear", lambda *a, **k: x.clone())
        m.setattr(net, "sla_gated_scan", lambda *a, **k: (x.clone(), x.clone(), x.clone()))
        d = fw.make_dual(x, torch.ones_like(x))
        for call in (lambda: net._Linear.apply(d, x, x, x, 0),
                     lambda: net._Linear.apply(x, x, x, d, 3),
                     lambda: net._GatedScan.apply(x, d, x, None, 1, True)):
            with pytest.raises(NotImplementedError):
                call()


def test_another_stream_gets_the_copies_and_the_memory_too(monkeypatch):
    """With stream= everything of an sla_* call happens on that stream."""
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

    def watched(make, what):
        def call(*a, **k):
            seen.append((what, inside[0]))
            return make(*a, **k)
        return call
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name), "memory"))
    monkeypatch.setattr(net, "_rows", watched(net._rows, "copy"))

    def kernel(*args):
        seen.append(("kernel", args[-1]))
        return 0
    names = ("sla_linear", "sla_linear_grad", "sla_gated_scan", "sla_gated_scan_grad",
             "sla_gated_scan_step", "sla_orthogonalise")
    monkeypatch.setattr(net, "_lib", types.SimpleNamespace(**{n: kernel for n in names}))
    monkeypatch.setattr(net, "_work_bytes", lambda *a: 64)
    monkeypatch.setattr(net, "_linear_bytes", lambda *a: (64, 64))
    monkeypatch.setattr(net, "_scan_dims", lambda *a: (dims(), None, 64, 64))
    x, w, y = torch.zeros(8, 4).t(), torch.zeros(16, 8), torch.zeros(16, 4).t()
    s, state = torch.zeros(2, 4, 24), torch.zeros(2, 24)
    calls = {
        "sla_linear": (x, w, None, y, 0),
        "sla_linear_grad": (y, x, w, None, 0, True, True, True, None),
        "sla_gated_scan": (s, s, None, state, 2, True, True),
        "sla_gated_scan_grad": (s, s, s, s, state, 2, False, True, True, True),
        "sla_gated_scan_step": (s[:, 0], s[:, 0], state),
        "sla_orthogonalise": (x, 1, ((1.0, 0.0, 0.0),), 1e-7),
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
    monkeypatch.setattr(net, "_lib", types.SimpleNamespace(sla_gated_scan_step=lambda *a: 0))
    monkeypatch.setattr(net, "_scan_dims", lambda *a: (dims(), None, 64, 64))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    x = torch.zeros(2, 4)
    leaf = torch.randn(2, 4, requires_grad=True)
    state = leaf.clone()
    loss = state.square().sum()
    net.sla_gated_scan_step(x, x, state.detach())
    assert state._version == 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_what_the_forward_pass_keeps_is_small():
    """A state for every block of tokens, and the workspaces stay proportional to the tensors."""
    n, m = K._I64(), K._I64()
    for seqs, tokens, channels, packed in ((4, 16384, 2048, 0), (1, 1 << 20, 16, 0),
                                           (100000, 100000, 64, 1), (23, 12345, 999, 1)):
        d = dims(sequences=seqs, tokens=tokens, channels=channels, packed=packed)
        assert lib.sla_gated_scan_work(ctypes.byref(d), ctypes.byref(n), ctypes.byref(m)) == K.OK
        assert n.value <= 4 * channels * (tokens / 8 + 2 * seqs) + 4 * seqs + 1024
        assert m.value <= 8 * 64 * seqs * channels + 4 * seqs + 1024
