"""Network operators on the library's kernels: layer norm, the gated
feed-forward unit, and the gated delta rule (whole sequences, and single
tokens against a kept state).

They are the parts of a network that predicts a system's coefficients and is
trained through the solver's adjoint (``examples/coefficient_network.py``).
As everywhere in this package a function marshals its arguments and calls the
C ABI of the same name (``include/sla.h``); the autograd nodes stand on top.
Work is enqueued on the current stream, workspaces come from PyTorch's
allocator on that stream, nothing synchronises (but offsets given on the host,
which are copied), and the same inputs give the same bits.  The sla_* functions
take another stream too: everything they do then happens on it, so it has to be
ordered behind the inputs, which live until it is done, and what is returned
belongs to it.

Inputs may be views whose last axis is contiguous and whose rows (tokens) are
evenly spaced, such as the parts of one fused projection; any other layout is
copied first.  Types: float32, float16 and bfloat16, with sums, statistics
and states in float32.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math

import torch
import torch.autograd.forward_ad as forward_ad
from torch.autograd.function import once_differentiable

from . import _I64, _check, _lib

F32, F16, BF16 = 0, 1, 2
_TYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


class _DeltaDims(ctypes.Structure):
    _fields_ = [("sequences", _I64), ("tokens", _I64), ("key_heads", _I64),
                ("value_heads", _I64), ("key_dim", _I64), ("value_dim", _I64),
                ("scale", ctypes.c_double), ("type", ctypes.c_int), ("packed", ctypes.c_int)]


def _tensor(t, name: str, like: torch.Tensor | None = None, dtypes=None) -> torch.Tensor:
    """Refuses what no kernel takes: other types, other devices than `like`'s."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a GPU tensor (the library has no CPU path)")
    if like is None:
        if t.get_device() != torch._C._cuda_getDevice():
            raise ValueError(f"{name}: is on {t.device}, which is not the current device")
    elif t.get_device() != like.get_device():
        raise ValueError(f"{name}: is on {t.device}, the other tensors on {like.device}")
    if t.dtype not in (dtypes or _TYPES):
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes or _TYPES)}, "
                        f"got {t.dtype}")
    return t


def _stream(like: torch.Tensor) -> int:
    """The raw current stream of like's device.  (The stream object of
    torch.cuda costs as much as a launch.)"""
    return torch._C._cuda_getCurrentRawStream(like.get_device())


def _takes_stream(f):
    """f(..., stream=None): all of f on that stream (a torch stream or a raw
    one), its copies and allocations included.  Memory of another stream's pool
    would be given out again while the kernels still use it."""
    signature = inspect.signature(f)
    known = [*signature.parameters.values()]
    extra = inspect.Parameter("stream", inspect.Parameter.POSITIONAL_OR_KEYWORD, default=None)

    @functools.wraps(f)
    def call(*args, **kwargs):
        stream = kwargs.pop("stream", None)
        if len(args) > len(known):
            *args, stream = args
        if stream is None:
            return f(*args, **kwargs)
        if not hasattr(stream, "cuda_stream"):
            device = next(t for t in (*args, *kwargs.values())
                          if isinstance(t, torch.Tensor)).device
            stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) \
                else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            return f(*args, **kwargs)
    call.__signature__ = signature.replace(parameters=[*known, extra])
    return call


@functools.lru_cache(maxsize=1024)
def _work_bytes(entry: str, *args) -> int:
    """What a workspace call says; the sizes alone decide it."""
    n = _I64()
    _check(getattr(_lib, entry)(*args, ctypes.byref(n)))
    return n.value


def _sized(t: torch.Tensor, shape: tuple, name: str):
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t: torch.Tensor, tail: int):
    """(t, elements from one row to the next): the last `tail` axes are a row,
    contiguous in itself; the axes before it are the rows.  t is copied if its
    rows are not evenly spaced."""
    width = 1
    for n in t.shape[t.dim() - tail:]:
        width *= n
    if t.is_contiguous():
        return t, width
    lead = t.dim() - tail
    want = 1
    for n, s in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        if n != 1 and s != want:
            t = t.contiguous()
            return t, width
        want *= n
    step, count = None, 1
    for n, s in zip(reversed(t.shape[:lead]), reversed(t.stride()[:lead])):
        if n == 1:
            continue
        if step is None:
            step = s
        if s != step * count or step < width:
            t = t.contiguous()
            return t, width
        count *= n
    return t, max(step or width, width)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _wants(*tensors) -> bool:
    """Whether a derivative is asked for: a gradient, or a tangent (which does
    not require grad and passes no_grad; the autograd nodes refuse it)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                return True
    return False


def _block(nbytes: int, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device)


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
@_takes_stream
def sla_layer_norm(x, weight, bias, eps: float, want_stats: bool = False):
    """(y, stats): stats [rows, 2] = mean less the row's first element and
    1 / sqrt(var + eps), or mean and -1 / sqrt(var + eps) if that lies nearer to
    zero; or None."""
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    x, ld = _rows(x, 1)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    stats = torch.empty(rows, 2, dtype=torch.float32, device=x.device) if want_stats else None
    par = weight if weight is not None else bias
    _check(_lib.sla_layer_norm(x.data_ptr(), ld, rows, cols, _TYPES[x.dtype], _ptr(weight),
                               _ptr(bias), _TYPES[par.dtype if par is not None else x.dtype],
                               eps, y.data_ptr(), _ptr(stats), _stream(x)))
    return y, stats


@_takes_stream
def sla_layer_norm_grad(dy, x, weight, stats, want_x=True, want_weight=True, want_bias=True,
                        wtype=None):
    """(dx, dweight, dbias), None where not wanted."""
    cols = x.shape[-1]
    rows = x.numel() // cols
    x, ldx = _rows(x, 1)
    dy, lddy = _rows(dy, 1)
    wtype = wtype or (weight.dtype if weight is not None else x.dtype)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if want_x else None
    dw = torch.empty(cols, dtype=wtype, device=x.device) if want_weight else None
    db = torch.empty(cols, dtype=wtype, device=x.device) if want_bias else None
    work, size = None, 0
    if want_weight or want_bias:
        size = _work_bytes("sla_layer_norm_work", rows, cols, _TYPES[x.dtype])
        work = _block(size, x)
    _check(_lib.sla_layer_norm_grad(dy.data_ptr(), lddy, x.data_ptr(), ldx, rows, cols,
                                    _TYPES[x.dtype], _ptr(weight), _TYPES[wtype],
                                    stats.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db), _ptr(work),
                                    size, _stream(x)))
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, stats = sla_layer_norm(x, weight, bias, eps, want_stats=True)
        ctx.wtype = weight.dtype if weight is not None else bias.dtype if bias is not None \
            else x.dtype
        ctx.save_for_backward(x, weight, stats)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        return (*sla_layer_norm_grad(dy, x, weight, stats, need[0], need[1], need[2],
                                     ctx.wtype), None)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5) -> torch.Tensor:
    """Layer norm over the last axis: (x - mean) / sqrt(var + eps) * weight + bias.

    x [..., cols] of any supported type; weight and bias [cols] of x's type or
    float32 (both alike), either may be None.  One autograd node; the gradient
    keeps mean and 1 / sqrt(var + eps) of each row."""
    _tensor(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x: expected [..., cols] with cols >= 1")
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _tensor(t, name, x, (x.dtype, torch.float32))
            _sized(t, x.shape[-1:], name)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same type")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    weight = None if weight is None else weight.contiguous()
    bias = None if bias is None else bias.contiguous()
    if _wants(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, float(eps))
    return sla_layer_norm(x, weight, bias, float(eps))[0]


# ---------------------------------------------------------------------------
# The gated feed-forward unit
# ---------------------------------------------------------------------------
@_takes_stream
def sla_gated_ffn(x, w_gate, w_up, act: int):
    """h [..., outer] = f(x w_gate^T) * (x w_up^T)."""
    outer, inner = w_gate.shape
    x, ld = _rows(x, 1)
    h = torch.empty((*x.shape[:-1], outer), dtype=x.dtype, device=x.device)
    _check(_lib.sla_gated_ffn(x.data_ptr(), ld, w_gate.data_ptr(), w_up.data_ptr(),
                              x.numel() // inner, inner, outer, _TYPES[x.dtype], act,
                              h.data_ptr(), _stream(x)))
    return h


@_takes_stream
def sla_gated_ffn_grad(dh, x, w_gate, w_up, act: int, want_x=True, want_w=True):
    """(dx, dw_gate, dw_up), None where not wanted."""
    outer, inner = w_gate.shape
    rows = x.numel() // inner
    x, ldx = _rows(x, 1)
    dh, lddh = _rows(dh, 1)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if want_x else None
    dwg = torch.empty_like(w_gate) if want_w else None
    dwu = torch.empty_like(w_up) if want_w else None
    size = _work_bytes("sla_gated_ffn_work", rows, inner, outer, _TYPES[x.dtype])
    work = _block(size, x)
    _check(_lib.sla_gated_ffn_grad(dh.data_ptr(), lddh, x.data_ptr(), ldx, w_gate.data_ptr(),
                                   w_up.data_ptr(), rows, inner, outer, _TYPES[x.dtype], act,
                                   _ptr(dx), _ptr(dwg), _ptr(dwu), work.data_ptr(), size,
                                   _stream(x)))
    return dx, dwg, dwu


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act):
        ctx.act = act
        ctx.save_for_backward(x, w_gate, w_up)
        return sla_gated_ffn(x, w_gate, w_up, act)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, w_gate, w_up = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dwg, dwu = sla_gated_ffn_grad(dh, x, w_gate, w_up, ctx.act, need[0],
                                          need[1] or need[2])
        return dx, dwg if need[1] else None, dwu if need[2] else None, None


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
              activation: str = "silu") -> torch.Tensor:
    """Gated feed-forward unit: h = f(x w_gate^T) * (x w_up^T).

    x [..., inner], the weights [outer, inner], all of one type; activation f:
    "silu", "gelu" (with erf) or "relu".  One autograd node that keeps only
    its inputs: backward computes both projections again, and rounds the
    gradients of both to x's type (fp16: times a power of two that keeps them
    in range) before the products that follow."""
    _tensor(x, "x")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    _tensor(w_gate, "w_gate", x, (x.dtype,))
    _tensor(w_up, "w_up", x, (x.dtype,))
    if w_gate.dim() != 2 or w_gate.shape[0] < 1 or w_gate.shape[1] < 1:
        raise ValueError("w_gate: expected [outer, inner]")
    _sized(w_up, w_gate.shape, "w_up")
    if x.dim() < 1 or x.shape[-1] != w_gate.shape[1]:
        raise ValueError(f"x: expected [..., {w_gate.shape[1]}], got {tuple(x.shape)}")
    act = ACTIVATIONS[activation]
    w_gate, w_up = w_gate.contiguous(), w_up.contiguous()
    if _wants(x, w_gate, w_up):
        return _GatedFFN.apply(x, w_gate, w_up, act)
    return sla_gated_ffn(x, w_gate, w_up, act)


# ---------------------------------------------------------------------------
# The gated delta rule
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def _dims(*args):
    """(the C structure, its address, the bytes that sla_delta_rule_work says)"""
    d = _DeltaDims(*args)
    kept, grad = _I64(), _I64()
    _check(_lib.sla_delta_rule_work(ctypes.byref(d), ctypes.byref(kept), ctypes.byref(grad)))
    return d, ctypes.byref(d), kept.value, grad.value


def _delta_dims(q, v, sequences, scale, packed):
    tokens = 1
    for n in q.shape[:-2]:
        tokens *= n
    return _dims(sequences, tokens, q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1],
                 scale, _TYPES[q.dtype], int(packed))


def _states(dims, like):
    return torch.empty(dims.sequences, dims.value_heads, dims.key_dim, dims.value_dim,
                       dtype=torch.float32, device=like.device)


@_takes_stream
def sla_delta_rule(q, k, v, g, beta, offsets, initial_state, sequences: int, scale: float,
                   want_state: bool = True):
    """(o, final_state or None, kept): kept is what the gradient reads."""
    dims, at, size, _ = _delta_dims(q, v, sequences, scale, offsets is not None)
    (q, ldq), (k, ldk), (v, ldv) = _rows(q, 2), _rows(k, 2), _rows(v, 2)
    kept = _block(size, q)
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    state = _states(dims, q) if want_state else None
    _check(_lib.sla_delta_rule(at, q.data_ptr(), ldq, k.data_ptr(), ldk,
                               v.data_ptr(), ldv, g.data_ptr(), beta.data_ptr(), _ptr(offsets),
                               _ptr(initial_state), o.data_ptr(), _ptr(state), kept.data_ptr(),
                               size, _stream(q)))
    return o, state, kept


@_takes_stream
def sla_delta_rule_grad(q, k, v, g, beta, kept, grad_o, grad_state, sequences: int, scale: float,
                        packed: bool, want_initial: bool = True):
    """(dq, dk, dv, dg, dbeta, grad of the initial state or None)."""
    dims, at, _, size = _delta_dims(q, v, sequences, scale, packed)
    (q, ldq), (k, ldk), (v, ldv) = _rows(q, 2), _rows(k, 2), _rows(v, 2)
    grad_o, ldo = _rows(grad_o, 2)
    work = _block(size, q)
    dq, dk, dv, dg, dbeta = (torch.empty(t.shape, dtype=t.dtype, device=t.device)
                             for t in (q, k, v, g, beta))
    ds0 = _states(dims, q) if want_initial else None
    _check(_lib.sla_delta_rule_grad(
        at, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, g.data_ptr(),
        beta.data_ptr(), kept.data_ptr(), kept.numel(), grad_o.data_ptr(), ldo, _ptr(grad_state),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _ptr(ds0),
        work.data_ptr(), size, _stream(q)))
    return dq, dk, dv, dg, dbeta, ds0


class _DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, offsets, sequences, scale, want_state):
        o, state, kept = sla_delta_rule(q, k, v, g, beta, offsets, initial_state, sequences,
                                        scale, want_state)
        ctx.sequences, ctx.scale, ctx.packed = sequences, scale, offsets is not None
        ctx.save_for_backward(q, k, v, g, beta, kept)
        ctx.set_materialize_grads(False)
        return o, state

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_o, grad_state):
        q, k, v, g, beta, kept = ctx.saved_tensors
        if grad_o is None:
            grad_o = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        if grad_state is not None:
            grad_state = grad_state.contiguous()
        grads = sla_delta_rule_grad(q, k, v, g, beta, kept, grad_o, grad_state, ctx.sequences,
                                    ctx.scale, ctx.packed, ctx.needs_input_grad[5])
        return (*[d if n else None for d, n in zip(grads, ctx.needs_input_grad)],
                None, None, None, None)


def _check_delta(q, k, v, g, beta, scale, lead: int):
    _tensor(q, "q")
    for t, name in ((k, "k"), (v, "v")):
        _tensor(t, name, q, (q.dtype,))
    for t, name in ((g, "g"), (beta, "beta")):
        _tensor(t, name, q, (torch.float32,))
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError(f"q, k and v: expected {lead + 2} axes (the last two: heads, features)")
    _sized(k, q.shape, "k")
    _sized(v, (*q.shape[:lead], v.shape[-2], v.shape[-1]), "v")
    _sized(g, v.shape[:-1], "g")
    _sized(beta, v.shape[:-1], "beta")
    if q.shape[-2] < 1 or v.shape[-2] < 1 or v.shape[-2] % q.shape[-2]:
        raise ValueError(f"v's heads ({v.shape[-2]}) must be a multiple of q's ({q.shape[-2]})")
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None and q.shape[-1] else scale
    if scale is None or not math.isfinite(scale):
        raise ValueError("scale must be finite")
    return float(scale)


def gated_delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     beta: torch.Tensor, scale: float | None = None,
                     initial_state: torch.Tensor | None = None,
                     output_final_state: bool = False, cu_seqlens=None):
    """The gated delta rule over whole sequences: (o, final state or None).

    Per head, with a state S [dk, dv]: S <- exp(g) S, then
    S <- S + k (beta (v - S^T k))^T, then o = scale S^T q.

    q, k [batch, tokens, heads, dk] (dk <= 128); v [batch, tokens, value_heads,
    dv], value_heads a multiple of heads (neighbouring value heads share a key
    head); g (log decay, <= 0; -inf or a type's lowest value begins the state
    anew, with a gradient of 0) and beta float32 [batch, tokens, value_heads].
    scale defaults to 1 / sqrt(dk).  States are float32 [sequences,
    value_heads, dk, dv]; without an initial state they begin at zero.

    With cu_seqlens the batch is 1 and sequence i is the tokens cu_seqlens[i]
    .. cu_seqlens[i+1] - 1: a list or CPU tensor is checked here and copied to
    the GPU, which waits for it; a GPU tensor (int32 or int64) is read by the
    kernels alone, which raise falling offsets and clamp those outside.  Tokens of no sequence get zeros.

    One autograd node, with gradients for q, k, v, g, beta and the initial
    state; it keeps the state before every chunk of 64 tokens.  A value that is
    not finite may spoil earlier tokens of its chunk of 64 too."""
    scale = _check_delta(q, k, v, g, beta, scale, 2)
    batch, tokens = q.shape[0], q.shape[1]
    offsets = None
    sequences = batch
    if cu_seqlens is not None:
        if batch != 1:
            raise ValueError("cu_seqlens needs a batch of 1")
        if not isinstance(cu_seqlens, torch.Tensor):
            cu_seqlens = torch.as_tensor(cu_seqlens)   # its own type: no rounding
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens: expected [sequences + 1]")
        if cu_seqlens.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"cu_seqlens: expected int32 or int64, got {cu_seqlens.dtype}")
        if not cu_seqlens.is_cuda:
            if bool((cu_seqlens.diff() < 0).any()) or int(cu_seqlens[0]) < 0 \
                    or int(cu_seqlens[-1]) > tokens:
                raise ValueError(f"cu_seqlens: offsets must not fall and lie in 0..{tokens}")
        elif cu_seqlens.device != q.device:
            raise ValueError(f"cu_seqlens: is on {cu_seqlens.device}, q on {q.device}")
        sequences = cu_seqlens.numel() - 1
        if cu_seqlens.dtype == torch.int64:  # clamped first: narrowing would wrap
            cu_seqlens = cu_seqlens.clamp(0, tokens)
        offsets = cu_seqlens.to(device=q.device, dtype=torch.int32).contiguous()
    if initial_state is not None:
        _tensor(initial_state, "initial_state", q, (torch.float32,))
        _sized(initial_state, (sequences, v.shape[2], q.shape[3], v.shape[3]), "initial_state")
        initial_state = initial_state.contiguous()
    g, beta = g.contiguous(), beta.contiguous()
    if _wants(q, k, v, g, beta, initial_state):
        return _DeltaRule.apply(q, k, v, g, beta, initial_state, offsets, sequences, scale,
                                bool(output_final_state))
    return sla_delta_rule(q, k, v, g, beta, offsets, initial_state, sequences, scale,
                          bool(output_final_state))[:2]


@_takes_stream
def sla_delta_step(q, k, v, g, beta, state, scale: float):
    """o [sequences, value_heads, dv]; state is updated in place."""
    at = _delta_dims(q, v, q.shape[0], scale, False)[1]
    (q, ldq), (k, ldk), (v, ldv) = _rows(q, 2), _rows(k, 2), _rows(v, 2)
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _check(_lib.sla_delta_step(at, q.data_ptr(), ldq, k.data_ptr(), ldk,
                               v.data_ptr(), ldv, g.data_ptr(), beta.data_ptr(),
                               state.data_ptr(), o.data_ptr(), _stream(q)))
    torch.autograd.graph.increment_version(state)  # a graph that saved it has to notice
    return o


def gated_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     beta: torch.Tensor, state: torch.Tensor,
                     scale: float | None = None) -> torch.Tensor:
    """One token of every sequence: o, with ``state`` updated in place.

    q, k [sequences, heads, dk], v [sequences, value_heads, dv], g and beta
    float32 [sequences, value_heads], state float32 [sequences, value_heads,
    dk, dv], contiguous, as gated_delta_rule returns it.  For serving: it has
    no derivative, and refuses inputs that ask for a gradient or carry a
    tangent."""
    scale = _check_delta(q, k, v, g, beta, scale, 1)
    _tensor(state, "state", q, (torch.float32,))
    _sized(state, (q.shape[0], v.shape[1], q.shape[2], v.shape[2]), "state")
    if not state.is_contiguous():
        raise ValueError("state: expected a contiguous tensor (it is updated in place)")
    if _wants(q, k, v, g, beta, state):
        raise ValueError("gated_delta_step has no gradient (and no tangent): use "
                         "gated_delta_rule, or no_grad and plain inputs")
    return sla_delta_step(q, k, v, g.contiguous(), beta.contiguous(), state, scale)
