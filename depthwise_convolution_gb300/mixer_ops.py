"""Python binding of the token mixer's entry points, one function per entry point, same names.

Argument marshalling only, like :mod:`ops`: PyTorch CUDA tensors in, kernels of
libdwconv on the current stream (or ``stream``) of the tensors' device.  Inputs
may be strided views (a slice of a wider projection) as long as their last
dimension is dense; outputs are dense.  Outputs and workspaces that the caller
does not pass are allocated on the stream the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch

from . import _lib
from .ops import _ll, _raw_stream

_FLOATS = {torch.float32: _lib.FP32, torch.float16: _lib.FP16, torch.bfloat16: _lib.BF16}
_ACTS = {"none": _lib.ACT_NONE, "silu": _lib.ACT_SILU}
NORMS = {"rms": _lib.NORM_RMS, "layer": _lib.NORM_LAYER}
GATES = {"none": _lib.GATE_NONE, "silu": _lib.GATE_SILU, "sigmoid": _lib.GATE_SIGMOID}
_HERE = contextlib.nullcontext()


_NATIVE = {}


@functools.lru_cache(maxsize=None)
def _module():
    return _lib.load_torch_ops()


def _native(name):
    """A function of libdwconv_torch.so.  It takes what the function here that calls it takes, with new outputs on the
    current stream, and returns NotImplemented for anything else, about which that function then has the words."""
    op = _NATIVE.get(name)
    if op is None:
        op = _NATIVE[name] = getattr(_module(), name)
    return op


def _choice(table, name, what):
    code = table.get(name)
    if code is None:
        raise ValueError(f"unknown {what} {name!r}; one of {sorted(table)}")
    return code


def _act(name):
    return _choice(_ACTS, name, "activation")


def _first(t, name):
    """(dtype code, device index) of the tensor that the others have to match."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code, t.get_device()


def _strided(t, name, shape, dev, dtype):
    """Address of a view whose last dimension is dense; checks its shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor" if not t.is_cuda else
                         f"{name} must be on cuda:{dev}, like the input")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return t.data_ptr()


def _dense(t, name, shape, dev, dtype):
    """Address of an optional dense tensor."""
    if t is None:
        return None
    p = _strided(t, name, shape, dev, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return p


# Metadata (shapes, strides, types, devices) that passed a function's checks, and
# the numbers it derives from them: a call that repeats them skips the checks.
# Addresses and values are not part of it.
_SEEN = {}
_MOST_SEEN = 4096


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _remember(key, value):
    if len(_SEEN) >= _MOST_SEEN:
        _SEEN.clear()
    _SEEN[key] = value
    return value


def _address(t):
    return None if t is None else t.data_ptr()


def _region(dev, stream):
    """Makes `dev` current, and memory allocated inside belong to the stream that the
    kernels run on, so that the caching allocator hands it out again only behind them."""
    if stream is None and dev == torch.cuda.current_device():
        return _HERE
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(dev))
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", dev))
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _current(dev):
    """The stream that _region made current."""
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


@functools.lru_cache(maxsize=1024)
def _longs(*values):
    return (ctypes.c_longlong * len(values))(*values)


def _written(t):
    """The caller's tensor is written in place: autograd has to see that."""
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _new(out, name, shape, dev, ref, dtype=None):
    """(tensor, address) of an output: the caller's, or a new one."""
    if out is None:
        out = torch.empty(shape, dtype=dtype or ref.dtype, device=ref.device)
        return out, out.data_ptr()
    p = _dense(out, name, shape, dev, dtype or ref.dtype)
    _written(out)
    return out, p


def _scratch(workspace, need, ref):
    """(workspace, address, bytes): the caller's, or one that is large enough, or none."""
    if workspace is not None:
        if not workspace.is_cuda or workspace.device != ref.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {ref.device}")
    elif need == 0:
        return None, None, 0
    else:
        workspace = torch.empty(need, dtype=torch.uint8, device=ref.device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _dtype_code(dtype) -> int:
    return dtype if isinstance(dtype, int) else _FLOATS[dtype]


# ---- causal convolution ----------------------------------------------------------------------------------------------

def _causal_checks(x, w, bias, ndim):
    dt, dev = _first(x, "x")
    if x.dim() != ndim:
        raise ValueError(f"x must have {ndim} dimensions, got {tuple(x.shape)}")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [W, C]")
    W, C = w.shape[0], x.shape[-1]
    _strided(x, "x", x.shape, dev, x.dtype)
    _dense(w, "w", (W, C), dev, x.dtype)
    _dense(bias, "bias", (C,), dev, torch.float32)
    return dt, dev, W, C


def _causal_sequence(x, w, bias, act, state, lengths):
    """The integers of a sequence call: (dt, dev, (B, T, C, W), act, x's strides)."""
    try:
        key = ("causal", act, _meta(x), _meta(w), _meta(bias), _meta(state), _meta(lengths))
        known = _SEEN.get(key)
    except AttributeError:
        known = key = None
    if known is not None:
        return known
    dt, dev, W, C = _causal_checks(x, w, bias, 3)
    B, T, _ = x.shape
    _dense(state, "state", (B, W - 1, C), dev, x.dtype)
    _dense(lengths, "lengths", (B,), dev, torch.int32)
    return _remember(key, (dt, dev, (B, T, C, W), _act(act), x.stride()[:2]))


def dwconv_causal_fwd(x, w, bias=None, act="silu", state=None, lengths=None, return_state=False, out=None,
                      state_out=None, stream=None):
    """y[b,t] = act(bias + sum_j w[j] x[b, t-(W-1)+j]).  x [B,T,C], w [W,C], bias [C]
    float32 or None, act "silu" or "none"; state [B,W-1,C] (the tokens before, None:
    zeros), lengths [B] int32 (right padding beyond) or None.  Returns y [B,T,C], with
    return_state (y, state_out): the window that the live tokens leave."""
    if out is None and state_out is None and stream is None:
        done = _native("causal_fwd")(x, w, bias, state, lengths, _act(act), bool(return_state))
        if done is not NotImplemented:
            return done if return_state else done[0]
    dt, dev, (B, T, C, W), code, xs = _causal_sequence(x, w, bias, act, state, lengths)
    with _region(dev, stream):
        out, op = _new(out, "out", (B, T, C), dev, x)
        sop = None
        if return_state or state_out is not None:
            state_out, sop = _new(state_out, "state_out", (B, W - 1, C), dev, x)
        _lib.check(_ll().dwconv_causal_fwd(B, T, C, W, dt, x.data_ptr(), *xs, w.data_ptr(), _address(bias), code,
                                           _address(state), _address(lengths), op, sop, _current(dev)),
                   "dwconv_causal_fwd")
    return (out, state_out) if return_state else out


@functools.lru_cache(maxsize=1024)
def _causal_bwd_bytes(B, T, C, W, code):
    return int(_ll().dwconv_causal_bwd_workspace_size(B, T, C, W, code))


def dwconv_causal_bwd_workspace_size(B, T, C, W, dtype) -> int:
    return _causal_bwd_bytes(B, T, C, W, _dtype_code(dtype))


def dwconv_causal_bwd(dy, x, w, bias=None, act="silu", state=None, lengths=None, need_db=True, need_dstate=False,
                      workspace=None, stream=None):
    """(dx [B,T,C], dw [W,C] float32, db [C] float32 or None, dstate [B,W-1,C] or None)
    of dwconv_causal_fwd for the gradient dy of its output."""
    dt, dev, (B, T, C, W), code, xs = _causal_sequence(x, w, bias, act, state, lengths)
    dyp = _strided(dy, "dy", (B, T, C), dev, x.dtype)
    with _region(dev, stream):
        dx, dxp = _new(None, "dx", (B, T, C), dev, x)
        dw, dwp = _new(None, "dw", (W, C), dev, x, torch.float32)
        db, dbp = _new(None, "db", (C,), dev, x, torch.float32) if need_db else (None, None)
        ds, dsp = _new(None, "dstate", (B, W - 1, C), dev, x) if need_dstate else (None, None)
        ws, wsp, wsb = _scratch(workspace, _causal_bwd_bytes(B, T, C, W, dt), x)
        _lib.check(_ll().dwconv_causal_bwd(
            B, T, C, W, dt, dyp, dy.stride(0), dy.stride(1), x.data_ptr(), *xs, w.data_ptr(), _address(bias), code,
            _address(state), _address(lengths), dxp, dwp, dbp, dsp, wsp, wsb, _current(dev)), "dwconv_causal_bwd")
    return dx, dw, db, ds


def dwconv_causal_step(x, w, state, bias=None, act="silu", slots=None, out=None, stream=None):
    """One token per row: x [B,C] against the windows state [N,W-1,C], shifted in place;
    slots [B] int32 names each row's window (None: its own row; outside [0,N): the row
    is idle and gives zeros).  Returns y [B,C]."""
    if out is None and stream is None:
        done = _native("causal_step")(x, w, state, bias, slots, _act(act))
        if done is not NotImplemented:
            return done
    try:
        key = ("causal step", act, _meta(x), _meta(w), _meta(state), _meta(bias), _meta(slots))
        known = _SEEN.get(key)
    except AttributeError:
        known = key = None
    if known is None:
        dt, dev, W, C = _causal_checks(x, w, bias, 2)
        if not isinstance(state, torch.Tensor) or state.dim() != 3:
            raise ValueError("state must be [N, W-1, C]")
        _dense(state, "state", (state.shape[0], W - 1, C), dev, x.dtype)
        _dense(slots, "slots", (x.shape[0],), dev, torch.int32)
        known = _remember(key, (dt, dev, (x.shape[0], state.shape[0], C, W), _act(act), x.stride(0)))
    dt, dev, (B, N, C, W), code, xs = known
    with _region(dev, stream):
        out, op = _new(out, "out", (B, C), dev, x)
        _lib.check(_ll().dwconv_causal_step(B, N, C, W, dt, x.data_ptr(), xs, w.data_ptr(), _address(bias), code,
                                            state.data_ptr(), _address(slots), op, _current(dev)),
                   "dwconv_causal_step")
    _written(state)
    return out


# ---- norms around a block --------------------------------------------------------------------------------------------

def _rows(t, name):
    """(outer stride, inner stride) of the rows of t [..., R, C]: the dimensions before
    the last two have to collapse into one."""
    C = t.shape[-1]
    inner = t.stride(-2) if t.dim() > 1 and t.shape[-2] > 1 else C
    outer, span = None, None
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        if outer is None:
            outer, span = s, n * s
        elif s == span:
            span = n * s
        else:
            raise ValueError(f"{name}: the dimensions before the last two must be collapsible (got strides "
                             f"{tuple(t.stride())})")
    return (inner * (t.shape[-2] if t.dim() > 1 else 1) if outer is None else outer), inner


def _norm_checks(tensors, weights, kind, gate_act):
    """The integers of a norm call: (dt, dev, outer, inner, C, strides or None, norm, gate).
    tensors: (y, name), ... of one shape and type; weights: (vector, name), ..."""
    try:
        key = ("norm", kind, gate_act, *[_meta(t) for t, _ in tensors], *[_meta(v) for v, _ in weights])
        known = _SEEN.get(key)
    except AttributeError:
        known = key = None
    if known is not None:
        return known
    y = tensors[0][0]
    dt, dev = _first(y, "y")
    if y.dim() < 1:
        raise ValueError("y must have at least one dimension")
    shape, dtype = y.shape, y.dtype
    C = shape[-1]
    inner = shape[-2] if len(shape) > 1 else 1
    outer = math.prod(shape[:-2])
    if inner == 0:
        outer, inner = 0, 1
    strides, dense = [], True
    for t, name in tensors:
        if t is None:
            strides += (0, 0)
            continue
        _strided(t, name, shape, dev, dtype)
        if t.is_contiguous():
            strides += (inner * C, C)
        else:
            strides += _rows(t, name)
            dense = False
    for v, name in weights:
        _dense(v, name, (C,), dev, torch.float32)
    return _remember(key, (dt, dev, outer, inner, C, None if dense else _longs(*strides),
                           _choice(NORMS, kind, "norm"), _choice(GATES, gate_act, "gate activation")))


def dwconv_block_norm_fwd(y, residual=None, gate=None, w_post=None, scale=None, w_pre=None, kind="rms",
                          gate_act="silu", eps=1e-6, stream=None):
    """h = residual + scale * post(y) * act(gate) and n = pre(h) over the last dimension.
    y, residual, gate [..., C]; w_post, scale, w_pre [C] float32; every part but y may be
    None (no norm after the block, no gate, scale 1, no residual, no norm of h).  kind
    "rms" or "layer", gate_act "silu", "sigmoid" or "none".  Returns (h, n), n None
    without w_pre."""
    if stream is None:
        done = _native("block_norm_fwd")(y, residual, gate, w_post, scale, w_pre, _choice(NORMS, kind, "norm"),
                                         _choice(GATES, gate_act, "gate activation"), eps)
        if done is not NotImplemented:
            return (done[0], done[1] if w_pre is not None else None)
    dt, dev, outer, inner, C, strides, norm, act = _norm_checks(
        ((y, "y"), (residual, "residual"), (gate, "gate")), ((w_post, "w_post"), (scale, "scale"), (w_pre, "w_pre")),
        kind, gate_act)
    with _region(dev, stream):
        h, hp = _new(None, "h", y.shape, dev, y)
        n, np = _new(None, "n", y.shape, dev, y) if w_pre is not None else (None, None)
        _lib.check(_ll().dwconv_block_norm_fwd(
            outer, inner, C, dt, norm, act, eps, y.data_ptr(), _address(residual), _address(gate), strides,
            _address(w_post), _address(scale), _address(w_pre), hp, np, _current(dev)), "dwconv_block_norm_fwd")
    return h, n


@functools.lru_cache(maxsize=1024)
def _norm_bwd_bytes(outer, inner, C, code):
    return int(_ll().dwconv_block_norm_bwd_workspace_size(outer, inner, C, code))


def dwconv_block_norm_bwd(dh, dn, y, residual=None, gate=None, w_post=None, scale=None, w_pre=None, kind="rms",
                          gate_act="silu", eps=1e-6, workspace=None, stream=None):
    """Gradients of dwconv_block_norm_fwd from dh and dn (either may be None): (dy,
    dresidual, dgate, dw_post, dscale, dw_pre), the weights' [C] float32, None for
    absent parts."""
    dt, dev, outer, inner, C, strides, norm, act = _norm_checks(
        ((y, "y"), (residual, "residual"), (gate, "gate"), (dh, "dh"), (dn, "dn")),
        ((w_post, "w_post"), (scale, "scale"), (w_pre, "w_pre")), kind, gate_act)
    with _region(dev, stream):
        outs = [(None, None) if t is None else _new(None, "", t.shape, dev, t)
                for t in (y, residual, gate, w_post, scale, w_pre)]
        ws, wsp, wsb = _scratch(workspace, _norm_bwd_bytes(outer, inner, C, dt), y)
        _lib.check(_ll().dwconv_block_norm_bwd(
            outer, inner, C, dt, norm, act, eps, y.data_ptr(), _address(residual), _address(gate), _address(dh),
            _address(dn), strides, _address(w_post), _address(scale), _address(w_pre), *[p for _, p in outs], wsp, wsb,
            _current(dev)), "dwconv_block_norm_bwd")
    return tuple([t for t, _ in outs])


# ---- gated delta rule ------------------------------------------------------------------------------------------------

def _delta_checks(q, k, v, g, beta, lead, state, vector, others=()):
    """The integers of a call: (first dimensions, (Hk, Hv, K, V), dt, dev, gate's dt, strides).
    q, k [*lead, Hk, K], v [*lead, Hv, V], g, beta [*lead, Hv]; lead: 1 or 2 dimensions;
    state and others: (tensor, name) float32 [.., Hv, K, V]; vector: (tensor, name) int32 [B]."""
    try:
        key = ("delta", lead, _meta(q), _meta(k), _meta(v), _meta(g), _meta(beta), _meta(state), _meta(vector[0]),
               *[_meta(t) for t, _ in others])
        known = _SEEN.get(key)
    except AttributeError:
        known = key = None
    if known is not None:
        return known
    dt, dev = _first(q, "q")
    if q.dim() != lead + 2 or not isinstance(v, torch.Tensor) or v.dim() != lead + 2:
        raise ValueError(f"q and v must have {lead + 2} dimensions")
    shape, vshape, dtype = q.shape, v.shape, q.dtype
    (Hk, K), (Hv, V), first = shape[lead:], vshape[lead:], tuple(shape[:lead])
    if Hk == 0 or Hv % Hk:
        raise ValueError(f"the value heads must be a multiple of the key heads, got {Hv} and {Hk}")
    if not isinstance(g, torch.Tensor) or (g.dtype != dtype and g.dtype != torch.float32):
        raise ValueError(f"g must be {dtype} or torch.float32")
    _strided(q, "q", shape, dev, dtype)
    _strided(k, "k", shape, dev, dtype)
    _strided(v, "v", (*first, Hv, V), dev, dtype)
    gshape, gdtype = (*first, Hv), g.dtype
    for t, name in ((g, "g"), (beta, "beta")):
        if not isinstance(t, torch.Tensor) or t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev}, like the input")
        if t.shape != gshape or t.dtype != gdtype:
            raise ValueError(f"{name} must be {list(gshape)} {gdtype}, got {list(t.shape)} {t.dtype}")
    if lead == 1 and (not isinstance(state, torch.Tensor) or state.dim() != 4):
        raise ValueError("state must be [N, Hv, K, V]")
    rows = state.shape[0] if lead == 1 else first[0]
    for t, name in ((state, "state"), *others):
        _dense(t, name, (rows, Hv, K, V), dev, torch.float32)
    _dense(vector[0], vector[1], first[:1], dev, torch.int32)
    strides = (*q.stride()[:-1], *k.stride()[:-1], *v.stride()[:-1], *g.stride(), *beta.stride())
    return _remember(key, (first, (Hk, Hv, K, V), dt, dev, _FLOATS[gdtype], strides))


@functools.lru_cache(maxsize=256)
def _delta_sizes(*shape):
    """Workspace of the forward pass; `saved`; workspace of the backward pass without and with it."""
    lib = _ll()
    return (int(lib.dwconv_delta_fwd_workspace_size(*shape)), int(lib.dwconv_delta_saved_size(*shape)),
            int(lib.dwconv_delta_bwd_workspace_size(*shape, 0)), int(lib.dwconv_delta_bwd_workspace_size(*shape, 1)))


def dwconv_delta_saved_size(B, T, Hk, Hv, K, V, dtype) -> int:
    """Bytes of the buffer that carries a forward pass over to its backward pass."""
    return _delta_sizes(B, T, Hk, Hv, K, V, _dtype_code(dtype))[1]


def _saved(saved, dev, shape):
    if saved is None:
        return None
    if saved.numel() * saved.element_size() < _delta_sizes(*shape)[1]:
        raise ValueError("saved is smaller than dwconv_delta_saved_size")
    if saved.get_device() != dev or not saved.is_contiguous():
        raise ValueError(f"saved must be a contiguous tensor on cuda:{dev}")
    return saved.data_ptr()


def dwconv_delta_fwd(q, k, v, g, beta, scale=None, qk_norm=False, state=None, lengths=None, return_state=False,
                     out=None, state_out=None, saved=None, workspace=None, stream=None):
    """Gated delta rule over sequences: q, k [B,T,Hk,K], v [B,T,Hv,V], g (log decay; minus
    infinity resets the state) and beta [B,T,Hv] of q's dtype or float32; scale defaults to K**-0.5; qk_norm divides q and
    k by their norms.  state [B,Hv,K,V] float32 (None: zeros), lengths [B] int32.  Returns
    o [B,T,Hv,V], with return_state (o, state_out).  saved: a buffer of
    dwconv_delta_saved_size bytes that dwconv_delta_bwd can then take over."""
    (B, T), (Hk, Hv, K, V), dt, dev, gdt, strides = _delta_checks(q, k, v, g, beta, 2, state, (lengths, "lengths"))
    shape = (B, T, Hk, Hv, K, V, dt)
    with _region(dev, stream):
        out, op = _new(out, "out", (B, T, Hv, V), dev, q)
        sop = None
        if return_state or state_out is not None:
            state_out, sop = _new(state_out, "state_out", (B, Hv, K, V), dev, q, torch.float32)
        ws, wsp, wsb = _scratch(workspace, 0 if saved is not None else _delta_sizes(*shape)[0], q)
        _lib.check(_ll().dwconv_delta_fwd(
            B, T, Hk, Hv, K, V, dt, gdt, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _longs(*strides), K ** -0.5 if scale is None else scale, int(qk_norm), _address(state), _address(lengths),
            op, sop, _saved(saved, dev, shape), wsp, wsb, _current(dev)), "dwconv_delta_fwd")
    return (out, state_out) if return_state else out


def dwconv_delta_bwd(do, q, k, v, g, beta, scale=None, qk_norm=False, state=None, lengths=None, dstate_out=None,
                     need_dstate=False, saved=None, workspace=None, stream=None):
    """(dq, dk, dv, dg, dbeta, dstate or None) of dwconv_delta_fwd for the gradients do of
    its output and dstate_out [B,Hv,K,V] float32 of its last state (None: zero).  saved:
    the buffer that the forward call filled, or None (its pass is repeated)."""
    (B, T), (Hk, Hv, K, V), dt, dev, gdt, strides = _delta_checks(q, k, v, g, beta, 2, state, (lengths, "lengths"),
                                                                  ((dstate_out, "dstate_out"),))
    dop = _strided(do, "do", (B, T, Hv, V), dev, q.dtype)
    shape = (B, T, Hk, Hv, K, V, dt)
    with _region(dev, stream):
        grads = [_new(None, "", t.shape, dev, t) for t in (q, k, v, g, beta)]
        ds, dsp = _new(None, "", (B, Hv, K, V), dev, q, torch.float32) if need_dstate else (None, None)
        ws, wsp, wsb = _scratch(workspace, _delta_sizes(*shape)[2 if saved is None else 3], q)
        _lib.check(_ll().dwconv_delta_bwd(
            B, T, Hk, Hv, K, V, dt, gdt, dop, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _longs(*strides, *do.stride()[:3]), K ** -0.5 if scale is None else scale, int(qk_norm), _address(state),
            _address(lengths), _address(dstate_out), *[p for _, p in grads], dsp, _saved(saved, dev, shape), wsp, wsb, _current(dev)), "dwconv_delta_bwd")
    return (*[t for t, _ in grads], ds)


def dwconv_delta_step(q, k, v, g, beta, state, scale=None, qk_norm=False, slots=None, out=None, stream=None):
    """One token per row: q, k [B,Hk,K], v [B,Hv,V], g, beta [B,Hv] against the states
    state [N,Hv,K,V] float32, updated in place; slots as in dwconv_causal_step.  Returns
    o [B,Hv,V]."""
    if out is None and stream is None:
        done = _native("delta_step")(q, k, v, g, beta, state, slots, scale, bool(qk_norm))
        if done is not NotImplemented:
            return done
    (B,), (Hk, Hv, K, V), dt, dev, gdt, strides = _delta_checks(q, k, v, g, beta, 1, state, (slots, "slots"))
    with _region(dev, stream):
        out, op = _new(out, "out", (B, Hv, V), dev, q)
        _lib.check(_ll().dwconv_delta_step(
            B, state.shape[0], Hk, Hv, K, V, dt, gdt, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
            beta.data_ptr(), _longs(*strides), K ** -0.5 if scale is None else scale, int(qk_norm), state.data_ptr(),
            _address(slots), op, _current(dev)), "dwconv_delta_step")
    _written(state)
    return out
