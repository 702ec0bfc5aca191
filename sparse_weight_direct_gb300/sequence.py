"""Sequence operators beside the sparse convolution: the short causal
convolution, the selective state space scan, the gated linear recurrence, the
low-rank adapters of many requests, the norms before and after a block, and beam
search's selection with the pools of states that follow it (include/spconv.h has
their formulas).

Activations are channels-first, (N, C, L) with the positions contiguous: a 1x1
layer's (N, C, H, W) with L = H * W.  Batch and channel strides are free, so a
half of a projection's channels can be passed as it lies.  They are float32,
bfloat16 or float16, all of one call alike; weights, their gradients and the
scan's states are float32.

Like ``forward``, these calls only marshal pointers: every step runs in
libspconv.so, asynchronously on ``stream`` (a torch stream or its handle;
default: the current torch stream), and a wrong argument raises SpconvError
before any work is enqueued.  Like every torch operation, a call on another
stream waits for nothing: its inputs have to be ready there, and whoever reads
its outputs elsewhere waits for that stream.

No call records anything for autograd: an input that requires a gradient gives
an output that does not.  A training step calls the *_backward functions.
"""
from __future__ import annotations

import ctypes
import operator
import struct
from array import array

from . import _lib
from ._lib import SpconvError

_codes_of = {_lib._i32: "i", _lib._i64: "q", _lib._ptr: "P", ctypes.c_float: "f"}


def _packer(structure):
    """Packs an argument structure of include/spconv.h, all but the workspace and
    its bytes, in one go: filling a ctypes structure field by field costs more
    than a short kernel runs."""
    return struct.Struct("".join(_codes_of[t] for n, t in structure._fields_ if "workspace" not in n)).pack


_pack_conv, _pack_scan, _pack_adapter = (
    _packer(s) for s in (_lib.ShortConvArgs, _lib.ScanArgs, _lib.AdapterArgs))
_pack_gated, _pack_norm, _pack_beam, _pack_reorder = (
    _packer(s) for s in (_lib.GatedScanArgs, _lib.ResidualNormArgs, _lib.BeamSelectArgs, _lib.ReorderArgs))
_pack_workspace = struct.Struct("Pq").pack
_no_workspace = _pack_workspace(0, 0)

_torch = None


def _load():
    """torch and its types, on the first call (the package itself loads without)."""
    global _torch, _Tensor, _codes, _f32, _i32, _bool, _empty, _empty_like, _raw_stream, _current_device, _library
    import torch
    _Tensor, _empty, _empty_like = torch.Tensor, torch.empty, torch.empty_like
    _f32, _i32, _bool = torch.float32, torch.int32, torch.bool
    _codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _current_device = torch.cuda.current_device
    _library = _lib.lib()
    _torch = torch


def _fail(what):
    raise SpconvError(_lib.SPCONV_ERR_INVALID_ARG, what)


def _not_packed(error):
    _fail(f"a size or a flag of the call does not fit its 32 bits ({error})")


def _begin(t, name, dims):
    """The tensor that a call's others go by: its type, its code, its device."""
    if _torch is None:
        _load()
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dtype not in _codes or t.dim() != dims:
        _fail(f"{name} must be a float32, bfloat16 or float16 CUDA tensor with {dims} dimensions")
    if t.numel() >> 31 and max(t.shape) >> 31:  # (before anything of that size is allocated)
        _fail(f"{name} has a size that is not below 2^31")
    dtype, device = t.dtype, t.get_device()
    if device != _current_device():
        _fail(f"{name} must be on the current CUDA device")
    return dtype, _codes[dtype], device


def _rows(t, name, dtype, device, shape):
    """Pointer to and strides of an activation whose last dimension is contiguous."""
    if not isinstance(t, _Tensor) or t.dtype != dtype or t.get_device() != device or t.shape != shape:
        _fail(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on CUDA device {device}")
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1 and t.numel():
        _fail(f"{name} must be contiguous along its last dimension")
    return t.data_ptr(), strides


def _whole(t, name, dtype, device, shape):
    """Pointer to a contiguous tensor, 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or t.dtype != dtype or t.get_device() != device or t.shape != shape:
        _fail(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on CUDA device {device}")
    if not t.is_contiguous():
        _fail(f"{name} must be contiguous")
    return t.data_ptr()


def _new(shape, dtype, device):
    return _empty(shape, dtype=dtype, device=device)


def _like(t):
    """A new contiguous tensor of t's shape and type."""
    return _empty_like(t) if t.is_contiguous() else _empty(t.shape, dtype=t.dtype, device=t.device)


def _dims(t, count, name):
    if not isinstance(t, _Tensor) or t.dim() != count:
        _fail(f"{name} must be a tensor with {count} dimensions")
    return t.shape


def _run(function, args, device, query=None):
    """Enqueues a call on the current stream."""
    if query is not None:
        need = query(args + _no_workspace)
        if need:
            workspace = _empty(need, dtype=_torch.uint8, device=device)
        args += _pack_workspace(workspace.data_ptr(), need) if need else _no_workspace
    rc = function(args, _raw_stream(device))
    if rc:
        _lib.check(rc, function.__name__)


def _elsewhere(call, stream, given, named):
    """The call with `stream` as the current one, so that its outputs and its
    workspace come from memory that this stream's own work is done with: a block
    that was given back to the caller's stream may still be read there.  Its
    tensors are marked as used on the other of the two streams, so that their
    memory is not given out again before that has passed what it holds now."""
    if _torch is None:
        _load()
    if not any(isinstance(t, _Tensor) and t.is_cuda for t in given):
        return call(*given, **named)  # (refused)
    cuda = _torch.cuda
    current, on = cuda.current_stream(), stream
    if not isinstance(stream, cuda.Stream):
        ptr = stream if isinstance(stream, int) else stream.cuda_stream
        on = cuda.ExternalStream(ptr) if ptr else cuda.default_stream()
    if on.cuda_stream == current.cuda_stream:
        return call(*given, **named)
    with cuda.stream(on):
        result = call(*given, **named)
    for t in (*given, *named.values()):
        for t in t if isinstance(t, (list, tuple)) else (t,):
            if isinstance(t, _Tensor):
                t.record_stream(on)
    outputs = result.values() if isinstance(result, dict) else result if isinstance(result, tuple) else (result,)
    for t in outputs:
        if t is not None:
            t.record_stream(current)
    return result


def short_conv(x, weight, bias=None, *, silu: bool = True, state=None, final_state=None,
               lengths=None, out=None, stream=None):
    """Short causal convolution: y_t = act(bias + sum_k weight[:, k] *
    x_(t-K+1+k)) per channel, with ``state`` (or zeros) before the first
    position.  x: (N, C, L); weight: (C, K) float32, K = 1..4; bias: (C,)
    float32; state: (N, C, K-1), the inputs before x; lengths: (N,) int32, outputs behind
    them are zero; final_state (optional, same shape as state): overwritten
    with the state behind the last position.  Returns y (``out`` if given)."""
    if stream is not None:
        return _elsewhere(short_conv, stream, (x, weight, bias),
                          dict(silu=silu, state=state, final_state=final_state, lengths=lengths, out=out))
    dt, code, dev = _begin(x, "x", 3)
    shape = N, C, L = x.shape
    K = _dims(weight, 2, "weight")[1]
    st = (N, C, K - 1)
    x_at, (xn, xc, _) = _rows(x, "x", dt, dev, shape)
    if out is None:
        out = _like(x)
    try:
        args = _pack_conv(
            N, C, L, K, code, silu, 0, 0, xn, xc, 0, 0, x_at, _whole(weight, "weight", _f32, dev, (C, K)),
            _whole(bias, "bias", _f32, dev, (C,)), _whole(state, "state", dt, dev, st),
            _whole(lengths, "lengths", _i32, dev, (N,)), 0, _whole(out, "out", dt, dev, shape),
            _whole(final_state, "final_state", dt, dev, st), 0, 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_short_conv, args + _no_workspace, dev)
    return out


def short_conv_backward(dy, x, weight, bias=None, *, silu: bool = True, state=None,
                        dfinal_state=None, lengths=None, stream=None):
    """Gradients of ``short_conv`` called with the same arguments, from those of
    y (dy) and, optionally, of final_state: (dx, dweight, dbias, dstate), with
    None for dbias without a bias and for dstate without a state."""
    if stream is not None:
        return _elsewhere(short_conv_backward, stream, (dy, x, weight, bias),
                          dict(silu=silu, state=state, dfinal_state=dfinal_state, lengths=lengths))
    dt, code, dev = _begin(x, "x", 3)
    shape = N, C, L = x.shape
    K = _dims(weight, 2, "weight")[1]
    st = (N, C, K - 1)
    x_at, (xn, xc, _) = _rows(x, "x", dt, dev, shape)
    dy_at, (dyn, dyc, _) = _rows(dy, "dy", dt, dev, shape)
    dx, dw = _new(shape, dt, dev), _new((C, K), _f32, dev)
    db = _new((C,), _f32, dev) if bias is not None else None
    ds = _new(st, dt, dev) if state is not None else None
    try:
        args = _pack_conv(
            N, C, L, K, code, silu, 0, 0, xn, xc, dyn, dyc, x_at, _whole(weight, "weight", _f32, dev, (C, K)),
            _whole(bias, "bias", _f32, dev, (C,)), _whole(state, "state", dt, dev, st),
            _whole(lengths, "lengths", _i32, dev, (N,)), 0, 0, 0, 0, dy_at,
            _whole(dfinal_state, "dfinal_state", dt, dev, st), dx.data_ptr(),
            0 if ds is None else ds.data_ptr(), dw.data_ptr(), 0 if db is None else db.data_ptr())
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_short_conv_backward, args, dev,
         _library.spconv_short_conv_backward_workspace)
    return dx, dw, db, ds


def short_conv_step(x, state, weight, bias=None, *, silu: bool = True, slots=None, out=None,
                    stream=None):
    """One position of each of N requests: x (N, C) -> y (N, C), and ``state``
    (num_slots, C, K-1) moved on in place.  Request n uses state slots[n] ((N,)
    int32; None: number n); one whose slot is outside gets zeros and changes
    nothing."""
    if stream is not None:
        return _elsewhere(short_conv_step, stream, (x, state, weight, bias),
                          dict(silu=silu, slots=slots, out=out))
    dt, code, dev = _begin(x, "x", 2)
    shape = N, C = x.shape
    K = _dims(weight, 2, "weight")[1]
    pool = _dims(state, 3, "state")[0]
    x_at, (xn, _) = _rows(x, "x", dt, dev, shape)
    if out is None:
        out = _like(x)
    try:
        args = _pack_conv(
            N, C, 1, K, code, silu, pool, 0, xn, 1, 0, 0, x_at, _whole(weight, "weight", _f32, dev, (C, K)), _whole(bias, "bias", _f32, dev, (C,)), 0, 0,
            _whole(slots, "slots", _i32, dev, (N,)), _whole(out, "out", dt, dev, shape), 0,
            _whole(state, "state", dt, dev, (pool, C, K - 1)), 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_short_conv_step, args + _no_workspace, dev)
    return out


def _scan_inputs(dt, code, dev, u, delta, A, B, C, D, z, delta_bias, softplus, step, pool, dy=None):
    """What the scan's calls have in common, up to the pointer to delta_bias, S, and the pointer to dy.
    B and C: (N, S[, L]) or (N, groups, S[, L])."""
    shape = u.shape
    N, ch = shape[0], shape[1]
    L = 1 if step else shape[2]
    S = _dims(A, 2, "A")[1]
    dims = 3 if step else 4  # of grouped B and C
    G = 1
    if isinstance(B, _Tensor) and B.dim() == dims:
        G = B.shape[1]
        if G < 1 or ch % G:
            _fail("the groups of B and C must divide the channels")
    whole, plain = ((N, G, S), (N, S)) if step else ((N, G, S, L), (N, S, L))
    grouped_b = isinstance(B, _Tensor) and B.dim() == dims
    grouped_c = isinstance(C, _Tensor) and C.dim() == dims
    if G > 1 and not grouped_c:
        _fail("B and C must have the same groups")
    at_b, sb = _rows(B, "B", dt, dev, whole if grouped_b else plain)
    at_c, sc = _rows(C, "C", dt, dev, whole if grouped_c else plain)
    at_u, su = _rows(u, "u", dt, dev, shape)
    at_d, sd = _rows(delta, "delta", dt, dev, shape)
    at_z, sz = (0, (0, 0)) if z is None else _rows(z, "z", dt, dev, shape)
    at_dy, sy = (0, (0, 0)) if dy is None else _rows(dy, "dy", dt, dev, shape)
    bg, cg = sb[1] if grouped_b else 0, sc[1] if grouped_c else 0
    if step:
        strides = (su[0], 1, sd[0], 1, sz[0], 1, 0, 0, sb[0], bg, 1, sc[0], cg, 1)
    else:
        strides = (su[0], su[1], sd[0], sd[1], sz[0], sz[1], sy[0], sy[1], sb[0], bg, sb[-2], sc[0], cg,
                   sc[-2])
    return (N, ch, L, S, G, code, softplus, pool, *strides, at_u, at_d, at_z, at_b, at_c,
            _whole(A, "A", _f32, dev, (ch, S)), _whole(D, "D", _f32, dev, (ch,)),
            _whole(delta_bias, "delta_bias", _f32, dev, (ch,))), S, at_dy


def scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, *, softplus: bool = True, state=None,
         final_state=None, lengths=None, out=None, stream=None):
    """Selective state space scan.  u, delta, z: (N, channels, L); A: (channels,
    S) float32, S = 1..64; B, C: (N, S, L) or (N, groups, S, L); D, delta_bias:
    (channels,) float32; state: (N, channels, S) float32, zeros if None.

        dt = softplus(delta + delta_bias)          (softplus=False: without it)
        h_t = exp(dt A) h_(t-1) + dt u_t B_t
        y_t = (C_t . h_t + D u_t) * z_t sigmoid(z_t)

    lengths: (N,) int32, outputs behind them are zero; final_state (optional):
    overwritten with h behind the last position.  Returns y."""
    if stream is not None:
        return _elsewhere(scan, stream, (u, delta, A, B, C, D, z, delta_bias),
                          dict(softplus=softplus, state=state, final_state=final_state, lengths=lengths, out=out))
    dt, code, dev = _begin(u, "u", 3)
    shape = u.shape
    given, S, _ = _scan_inputs(dt, code, dev, u, delta, A, B, C, D, z, delta_bias, softplus, False, 0)
    states = (shape[0], shape[1], S)
    if out is None:
        out = _like(u)
    try:
        args = _pack_scan(
            *given, _whole(state, "state", _f32, dev, states),
            _whole(lengths, "lengths", _i32, dev, shape[:1]), 0, _whole(out, "out", dt, dev, shape),
            _whole(final_state, "final_state", _f32, dev, states), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_scan, args, dev,
         _library.spconv_scan_workspace)
    return out


def scan_backward(dy, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, softplus: bool = True,
                  state=None, dfinal_state=None, lengths=None, stream=None) -> dict:
    """Gradients of ``scan`` called with the same arguments, from those of y (dy)
    and, optionally, of final_state: a dict of du, ddelta, dA, dB, dC, dD, dz,
    ddelta_bias and dstate, None for an argument that was not given."""
    if stream is not None:
        return _elsewhere(scan_backward, stream, (dy, u, delta, A, B, C, D, z, delta_bias),
                          dict(softplus=softplus, state=state, dfinal_state=dfinal_state, lengths=lengths))
    dt, code, dev = _begin(u, "u", 3)
    shape = u.shape
    if dy is None:
        _fail("dy must be given")
    given, S, dy_at = _scan_inputs(dt, code, dev, u, delta, A, B, C, D, z, delta_bias, softplus,
                                   False, 0, dy)
    states = (shape[0], shape[1], S)
    g = dict(du=_new(shape, dt, dev), ddelta=_new(shape, dt, dev), dA=_new(A.shape, _f32, dev),
             dB=_new(B.shape, dt, dev), dC=_new(C.shape, dt, dev),
             dD=None if D is None else _new(D.shape, _f32, dev),
             dz=None if z is None else _new(shape, dt, dev),
             ddelta_bias=None if delta_bias is None else _new(delta_bias.shape, _f32, dev),
             dstate=None if state is None else _new(states, _f32, dev))
    at = {k: 0 if t is None else t.data_ptr() for k, t in g.items()}
    try:
        args = _pack_scan(
            *given, _whole(state, "state", _f32, dev, states),
            _whole(lengths, "lengths", _i32, dev, shape[:1]), 0, 0, 0, 0, dy_at,
            _whole(dfinal_state, "dfinal_state", _f32, dev, states), at["du"], at["ddelta"], at["dz"],
            at["dB"], at["dC"], at["dA"], at["dD"], at["ddelta_bias"], at["dstate"])
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_scan_backward, args, dev,
         _library.spconv_scan_backward_workspace)
    return g


def scan_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, softplus: bool = True,
              slots=None, out=None, stream=None):
    """One position of each of N requests: u, delta, z (N, channels), B and C
    (N, S) or (N, groups, S) -> y (N, channels); ``state`` (num_slots,
    channels, S) float32 is moved on in place.  slots as for
    ``short_conv_step``."""
    if stream is not None:
        return _elsewhere(scan_step, stream, (state, u, delta, A, B, C, D, z, delta_bias),
                          dict(softplus=softplus, slots=slots, out=out))
    dt, code, dev = _begin(u, "u", 2)
    shape = N, ch = u.shape
    pool = _dims(state, 3, "state")[0]
    given, S, _ = _scan_inputs(dt, code, dev, u, delta, A, B, C, D, z, delta_bias, softplus, True, pool)
    if out is None:
        out = _like(u)
    try:
        args = _pack_scan(
            *given, 0, 0, _whole(slots, "slots", _i32, dev, (N,)), _whole(out, "out", dt, dev, shape),
            0, _whole(state, "state", _f32, dev, (pool, ch, S)), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_scan_step, args + _no_workspace, dev)
    return out


def adapter_add(y, x, a, b, index, *, scale=None, out=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection: out[n] =
    y[n] + scale[i] * b[i] (a[i] x[n]) with i = index[n]; out[n] = y[n] where i
    is no adapter (-1).  x: (N, C, P) or, for single tokens, (N, C); y: the
    projection's output, (N, M, P) or (N, M); a: (adapters, R, C) and b:
    (adapters, M, R) of x's type, R = 1..64; index: (N,) int32; scale:
    (adapters,) float32, 1 if None.  out may be y itself.  Returns out.

    Sums are float32.  Prompts (P > 1) use matrix instructions: float32 factors
    are good to 2^-21 of each product there, 16-bit ones are whole
    (include/spconv.h)."""
    if stream is not None:
        return _elsewhere(adapter_add, stream, (y, x, a, b, index), dict(scale=scale, out=out))
    single = getattr(x, "ndim", 0) == 2
    dt, code, dev = _begin(x, "x", 2 if single else 3)
    N, C = x.shape[0], x.shape[1]
    P = 1 if single else x.shape[2]
    K, R, _ = _dims(a, 3, "a")
    M = _dims(b, 3, "b")[1]
    shape = (N, M) if single else (N, M, P)
    if y is None:
        _fail("y must be given")
    y_at = _whole(y, "y", dt, dev, shape)
    x_at, xs = _rows(x, "x", dt, dev, x.shape)
    if out is None:
        out = _like(y)
    try:
        args = _pack_adapter(
            N, P, C, M, R, K, code, 0, xs[0], xs[1], x_at, _whole(a, "a", dt, dev, (K, R, C)), _whole(b, "b", dt, dev, (K, M, R)),
            _whole(index, "index", _i32, dev, (N,)), _whole(scale, "scale", _f32, dev, (K,)), y_at,
            _whole(out, "out", dt, dev, shape))
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_adapter_add, args, dev)
    return out

def _gated_inputs(dt, code, dev, x, r, A, i, z, r_bias, i_bias, pool, dy=None):
    """What the gated recurrence's calls have in common, up to the pointer to i_bias, and the pointer to dy."""
    shape = x.shape
    N, ch = shape[0], shape[1]
    if i is None and i_bias is not None:
        _fail("i_bias belongs to i, which is not given")
    at_x, sx = _rows(x, "x", dt, dev, shape)
    at_r, sr = _rows(r, "r", dt, dev, shape)
    at_i, si = (0, (0, 0)) if i is None else _rows(i, "i", dt, dev, shape)
    at_z, sz = (0, (0, 0)) if z is None else _rows(z, "z", dt, dev, shape)
    at_dy, sy = (0, (0, 0)) if dy is None else _rows(dy, "dy", dt, dev, shape)
    if len(shape) == 2:
        L, strides = 1, (sx[0], 1, sr[0], 1, si[0], 1, sz[0], 1, 0, 0)
    else:
        L, strides = shape[2], (sx[0], sx[1], sr[0], sr[1], si[0], si[1], sz[0], sz[1], sy[0], sy[1])
    if A is None:
        _fail("A must be given")
    row = (ch,)
    return (N, ch, L, code, pool, 0, *strides, at_x, at_r, at_i, at_z, _whole(A, "A", _f32, dev, row),
            _whole(r_bias, "r_bias", _f32, dev, row), _whole(i_bias, "i_bias", _f32, dev, row)), at_dy


def gated_scan(x, r, A, i=None, z=None, r_bias=None, i_bias=None, *, state=None, final_state=None,
               lengths=None, out=None, stream=None):
    """Gated linear recurrence, one state for each channel.  x, r, i, z: (N,
    channels, L); A, r_bias, i_bias: (channels,) float32, A <= 0; state: (N,
    channels) float32, zeros if None.

        a_t = exp(A sigmoid(r_t + r_bias))
        h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t     (without i: x_t)
        y_t = h_t * z_t sigmoid(z_t)                                      (without z: h_t)

    lengths: (N,) int32, outputs behind them are zero; final_state (optional):
    overwritten with h behind the last position.  Returns y."""
    if stream is not None:
        return _elsewhere(gated_scan, stream, (x, r, A, i, z, r_bias, i_bias),
                          dict(state=state, final_state=final_state, lengths=lengths, out=out))
    dt, code, dev = _begin(x, "x", 3)
    shape = x.shape
    given, _ = _gated_inputs(dt, code, dev, x, r, A, i, z, r_bias, i_bias, 0)
    if out is None:
        out = _like(x)
    try:
        args = _pack_gated(
            *given, _whole(state, "state", _f32, dev, shape[:2]),
            _whole(lengths, "lengths", _i32, dev, shape[:1]), 0, _whole(out, "out", dt, dev, shape),
            _whole(final_state, "final_state", _f32, dev, shape[:2]), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_gated_scan, args + _no_workspace, dev)
    return out


def gated_scan_backward(dy, x, r, A, i=None, z=None, r_bias=None, i_bias=None, *, state=None,
                        dfinal_state=None, lengths=None, stream=None) -> dict:
    """Gradients of ``gated_scan`` called with the same arguments, from those of y
    (dy) and, optionally, of final_state: a dict of dx, dr, dA, di, dz, dr_bias,
    di_bias and dstate, None for an argument that was not given."""
    if stream is not None:
        return _elsewhere(gated_scan_backward, stream, (dy, x, r, A, i, z, r_bias, i_bias),
                          dict(state=state, dfinal_state=dfinal_state, lengths=lengths))
    dt, code, dev = _begin(x, "x", 3)
    shape = x.shape
    if dy is None:
        _fail("dy must be given")
    given, dy_at = _gated_inputs(dt, code, dev, x, r, A, i, z, r_bias, i_bias, 0, dy)
    row, states = shape[1:2], shape[:2]
    g = dict(dx=_new(shape, dt, dev), dr=_new(shape, dt, dev), dA=_new(row, _f32, dev),
             di=None if i is None else _new(shape, dt, dev), dz=None if z is None else _new(shape, dt, dev),
             dr_bias=None if r_bias is None else _new(row, _f32, dev),
             di_bias=None if i_bias is None else _new(row, _f32, dev),
             dstate=None if state is None else _new(states, _f32, dev))
    at = {k: 0 if t is None else t.data_ptr() for k, t in g.items()}
    try:
        args = _pack_gated(
            *given, _whole(state, "state", _f32, dev, states),
            _whole(lengths, "lengths", _i32, dev, shape[:1]), 0, 0, 0, 0, dy_at,
            _whole(dfinal_state, "dfinal_state", _f32, dev, states), at["dx"], at["dr"], at["di"], at["dz"],
            at["dA"], at["dr_bias"], at["di_bias"], at["dstate"])
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_gated_scan_backward, args, dev,
         _library.spconv_gated_scan_backward_workspace)
    return g


def gated_scan_step(state, x, r, A, i=None, z=None, r_bias=None, i_bias=None, *, slots=None, out=None,
                    stream=None):
    """One position of each of N requests: x, r, i, z (N, channels) -> y (N,
    channels); ``state`` (num_slots, channels) float32 is moved on in place.
    slots as for ``short_conv_step``."""
    if stream is not None:
        return _elsewhere(gated_scan_step, stream, (state, x, r, A, i, z, r_bias, i_bias),
                          dict(slots=slots, out=out))
    dt, code, dev = _begin(x, "x", 2)
    shape = N, ch = x.shape
    pool = _dims(state, 2, "state")[0]
    given, _ = _gated_inputs(dt, code, dev, x, r, A, i, z, r_bias, i_bias, pool)
    if out is None:
        out = _like(x)
    try:
        args = _pack_gated(
            *given, 0, 0, _whole(slots, "slots", _i32, dev, (N,)), _whole(out, "out", dt, dev, shape), 0,
            _whole(state, "state", _f32, dev, (pool, ch)), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_gated_scan_step, args + _no_workspace, dev)
    return out


def _norm_inputs(x, y, z, post, scale, pre, eps, lengths, dims, dsum=None, dout=None):
    """What the norm's calls have in common, up to the pointer to lengths, the pointers to dsum and
    dout, and the type, device and shape."""
    some, name = (x, "x") if x is not None else (y, "y")
    dt, code, dev = _begin(some, name, dims or (2 if getattr(some, "ndim", 0) == 2 else 3))
    shape = some.shape
    single = len(shape) == 2
    if y is None and not (z is None and post is None and scale is None):
        _fail("z, post and scale belong to y, which is not given")
    if single and lengths is not None:
        _fail("lengths belong to sequences, (N, C, L)")
    ptrs, strides = [], []
    for t, n in ((x, "x"), (y, "y"), (z, "z"), (dsum, "dsum"), (dout, "dout")):
        at, s = (0, (0, 0)) if t is None else _rows(t, n, dt, dev, shape)
        ptrs.append(at)
        strides += (s[0], 1 if single else s[1])
    row = (shape[1],)
    return (shape[0], shape[1], 1 if single else shape[2], code, eps, 0, *strides, *ptrs[:3],
            _whole(post, "post", _f32, dev, row), _whole(scale, "scale", _f32, dev, row),
            _whole(pre, "pre", _f32, dev, row), _whole(lengths, "lengths", _i32, dev, shape[:1])), ptrs[3:], dt, dev, shape


def residual_norm(x, y=None, z=None, *, post=None, scale=None, pre=None, eps: float = 1e-6, lengths=None,
                  sum_out=None, out=None, stream=None):
    """The end of a block and the norm in front of the next: x (the residual
    stream), y (the block's output) and z (its gate) are (N, C, L) or, for single
    tokens, (N, C); x or y may be None; post, scale and pre are (C,) float32.

        b   = y z sigmoid(z)                        (without z: y)
        sum = x + scale * post * b / rms(b)         (without post: scale * b)
        out = pre * sum / rms(sum)

    with rms(v) = sqrt(mean of v^2 over the channels + eps).  lengths: (N,) int32,
    outputs behind them are zero.  Returns (sum, out): without y the sum is x
    itself, without pre out is None.  z alone without x and pre is a gated norm:
    residual_norm(None, y, z, post=w)[0]."""
    if stream is not None:
        return _elsewhere(residual_norm, stream, (x, y, z),
                          dict(post=post, scale=scale, pre=pre, eps=eps, lengths=lengths, sum_out=sum_out, out=out))
    given, _, dt, dev, shape = _norm_inputs(x, y, z, post, scale, pre, eps, lengths, 0)
    if y is None:
        if pre is None:
            _fail("pre or y must be given")
        if sum_out is not None:
            _fail("the sum without y is x itself")
    elif sum_out is None:
        sum_out = _new(shape, dt, dev)
    if pre is None:
        if out is not None:
            _fail("out belongs to pre, which is not given")
    elif out is None:
        out = _new(shape, dt, dev)
    try:
        args = _pack_norm(*given, _whole(sum_out, "sum_out", dt, dev, shape), _whole(out, "out", dt, dev, shape),
                          0, 0, 0, 0, 0, 0, 0, 0)
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_residual_norm, args + _no_workspace, dev)
    return (x if y is None else sum_out), out


def residual_norm_backward(dsum, dout, x, y=None, z=None, *, post=None, scale=None, pre=None, eps: float = 1e-6,
                           lengths=None, stream=None) -> dict:
    """Gradients of ``residual_norm`` called with the same arguments on (N, C, L),
    from those of sum (dsum, or None) and out (dout; None without pre): a dict of
    dx, dy, dz, dpost, dscale and dpre, None for an argument that was not given.
    Without y, dsum is what x gets beside its norm's gradient."""
    if stream is not None:
        return _elsewhere(residual_norm_backward, stream, (dsum, dout, x, y, z),
                          dict(post=post, scale=scale, pre=pre, eps=eps, lengths=lengths))
    if (pre is None) != (dout is None):
        _fail("dout belongs to pre: both or neither must be given")
    if y is None and pre is None:
        _fail("pre or y must be given")
    given, (dsum_at, dout_at), dt, dev, shape = _norm_inputs(x, y, z, post, scale, pre, eps, lengths, 3, dsum, dout)
    row = shape[1:2]
    g = dict(dx=None if x is None else _new(shape, dt, dev), dy=None if y is None else _new(shape, dt, dev),
             dz=None if z is None else _new(shape, dt, dev), dpost=None if post is None else _new(row, _f32, dev),
             dscale=None if scale is None else _new(row, _f32, dev), dpre=None if pre is None else _new(row, _f32, dev))
    try:
        args = _pack_norm(*given, 0, 0, dsum_at, dout_at, *(0 if t is None else t.data_ptr() for t in g.values()))
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_residual_norm_backward, args, dev,
         _library.spconv_residual_norm_backward_workspace)
    return g


def beam_select(logits, scores, *, beams=None, eos=None, ended=None, stream=None):
    """Beam search's selection: the ``beams`` (default: as many as there are, at
    most 32) best ways in which N requests' beams can go on.  logits: (N, B, V),
    the vocabulary contiguous; scores: (N, B) float32, the beams' log
    probabilities; ended: (N, B) bool, beams that go on with token ``eos`` at no
    cost.

    Returns (scores, tokens, parents, ended), (N, beams) each, best first: the
    new log probabilities (float32), the tokens taken and the beams they continue
    (int32), and which have ended (bool; None without eos).  Ties go to the lowest
    parent, then the lowest token.  Where fewer ways have any chance, the rest are
    beams of their own number with token 0 and a score of minus infinity."""
    if stream is not None:
        return _elsewhere(beam_select, stream, (logits, scores), dict(beams=beams, eos=eos, ended=ended))
    dt, code, dev = _begin(logits, "logits", 3)
    N, B, V = logits.shape
    try:
        K = B if beams is None else operator.index(beams)
        token = -1 if eos is None else operator.index(eos)
    except (TypeError, ValueError) as error:
        _fail(f"beams and eos must be whole numbers ({error})")
    if eos is None:
        if ended is not None:
            _fail("ended beams need eos")
    elif not 0 <= token < V:
        _fail("eos must be one of the vocabulary's tokens")
    if not 1 <= K <= 32:
        _fail("1 to 32 beams can be selected")
    if scores is None:
        _fail("scores must be given")
    at, strides = _rows(logits, "logits", dt, dev, logits.shape)
    chosen = (N, K)
    new_scores, tokens, parents = _new(chosen, _f32, dev), _new(chosen, _i32, dev), _new(chosen, _i32, dev)
    new_ended = _new(chosen, _bool, dev) if eos is not None else None
    try:
        args = _pack_beam(N, B, V, K, code, token, strides[0], strides[1], at, _whole(scores, "scores", _f32, dev, (N, B)),
                          _whole(ended, "ended", _bool, dev, (N, B)), new_scores.data_ptr(), tokens.data_ptr(),
                          parents.data_ptr(), 0 if new_ended is None else new_ended.data_ptr())
    except struct.error as error:
        _not_packed(error)
    _run(_library.spconv_beam_select, args, dev, _library.spconv_beam_select_workspace)
    return new_scores, tokens, parents, new_ended


def reorder_states(pools, parents, slots, *, stream=None):
    """Pools of states follow their beams.  pools: a tensor or a list of tensors
    (num_slots, ...) of any type, such as those of the *_step calls; parents,
    slots: (N, B) int32, the beam that each of a request's B (at most 32) beams
    goes on from and the slots in which their states lie, none of them twice.

    A parent's first beam stays in its slot; every other one gets the slot of a
    beam that nobody goes on from, and a copy of its parent's states in each
    pool.  Returns the new slots, (N, B); ``slots`` itself is left as it was."""
    if not isinstance(pools, (list, tuple)):
        pools = (pools,)
    if stream is not None:
        return _elsewhere(_reorder_states, stream, (parents, pools, slots), {})
    return _reorder_states(parents, pools, slots)


def _reorder_states(parents, pools, slots):
    if _torch is None:
        _load()
    N, B = _dims(parents, 2, "parents")
    dev = parents.get_device()
    if not parents.is_cuda or dev != _current_device():
        _fail("parents must be on the current CUDA device")
    count = -1
    at, sizes = [], []
    for t in pools:
        if not isinstance(t, _Tensor) or t.get_device() != dev or not t.dim() or not t.is_contiguous():
            _fail(f"pools must be contiguous tensors on CUDA device {dev}")
        if count < 0:
            count = t.shape[0]
        elif t.shape[0] != count:
            _fail("pools must have the same number of slots")
        at.append(t.data_ptr())
        sizes.append(t.numel() // count * t.element_size() if count else 0)
    at, sizes = array("Q", at), array("q", sizes)
    new_slots = _new((N, B), _i32, dev)
    try:
        args = _pack_reorder(N, B, len(at), max(count, 0), at.buffer_info()[0], sizes.buffer_info()[0],
                             _whole(parents, "parents", _i32, dev, (N, B)), _whole(slots, "slots", _i32, dev, (N, B)),
                             new_slots.data_ptr())
    except struct.error as error:
        _not_packed(error)
    if slots is None:
        _fail("slots must be given")
    _run(_library.spconv_reorder_states, args, dev)
    return new_slots
