"""Sequence operators beside the sparse convolution: the short causal
convolution, the selective state space scan and the low-rank adapters of many
requests (include/spconv.h has their formulas).

Activations are channels-first, (N, C, L) with the positions contiguous: a 1x1
layer's (N, C, H, W) with L = H * W.  Batch and channel strides are free, so a
half of a projection's channels can be passed as it lies.  They are float32,
bfloat16 or float16, all of one call alike; weights, their gradients and the
scan's states are float32.

Like ``forward``, these calls only marshal pointers: every step runs in
libspconv.so, asynchronously on ``stream`` (default: the current torch
stream), and a wrong argument raises SpconvError before any work is enqueued.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import AdapterArgs, ScanArgs, ShortConvArgs, SpconvError

_dtypes = {}


def _torch():
    import torch
    if not _dtypes:
        _dtypes.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    return torch


def _fail(what):
    raise SpconvError(_lib.SPCONV_ERR_INVALID_ARG, what)


class _Call:
    """Checks a call's tensors and enqueues it on a stream.  On a stream other
    than the current one the tensors are marked as used there, so that their
    memory is not given out again before the stream has passed the call."""

    def __init__(self, lead, name, stream):
        self.torch = torch = _torch()
        if not (isinstance(lead, torch.Tensor) and lead.is_cuda and lead.dtype in _dtypes):
            _fail(f"{name} must be a float32, bfloat16 or float16 CUDA tensor")
        self.device, self.dtype = lead.device, lead.dtype
        self.code = _dtypes[lead.dtype]
        if self.device.index != torch.cuda.current_device():
            _fail(f"{name} must be on the current CUDA device")
        current = torch.cuda.current_stream()
        if stream is None:
            self.ptr, self.other = current.cuda_stream, None
        elif isinstance(stream, int):
            self.ptr = stream
            self.other = (torch.cuda.ExternalStream(stream) if stream != current.cuda_stream and stream
                          else None)
        else:
            self.ptr = stream.cuda_stream
            self.other = stream if self.ptr != current.cuda_stream else None
        self.used = []

    def _one(self, t, name, shape, dtype):
        if not (isinstance(t, self.torch.Tensor) and t.dtype == dtype and t.device == self.device
                and t.shape == shape):
            _fail(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {self.device}")
        if self.other is not None:
            self.used.append(t)

    def rows(self, t, name, shape):
        """An activation whose last dimension is contiguous: its pointer (strides are the caller's)."""
        self._one(t, name, shape, self.dtype)
        if shape[-1] > 1 and t.stride(-1) != 1:
            _fail(f"{name} must be contiguous along its last dimension")
        return t.data_ptr()

    def whole(self, t, name, shape, dtype=None):
        """A contiguous tensor or None: its pointer."""
        if t is None:
            return None
        self._one(t, name, shape, dtype or self.dtype)
        if not t.is_contiguous():
            _fail(f"{name} must be contiguous")
        return t.data_ptr()

    def new(self, shape, dtype=None):
        t = self.torch.empty(shape, dtype=dtype or self.dtype, device=self.device)
        if self.other is not None:
            self.used.append(t)
        return t

    def out(self, t, name, shape):
        if t is None:
            return self.new(shape)
        self.whole(t, name, shape)
        return t

    def workspace(self, args, function):
        need = getattr(_lib.lib(), function)(ctypes.byref(args))
        if need:
            t = self.new((need,), self.torch.uint8)
            args.workspace, args.workspace_bytes = t.data_ptr(), need
            return t  # kept until the launches are enqueued
        return None

    def run(self, function, args):
        rc = getattr(_lib.lib(), function)(ctypes.byref(args), self.ptr)
        if rc:
            _lib.check(rc, function)
        for t in self.used:
            t.record_stream(self.other)


def _dims(t, count, name):
    if getattr(t, "dim", lambda: -1)() != count:
        _fail(f"{name} must have {count} dimensions")
    return t.shape


def short_conv(x, weight, bias=None, *, silu: bool = True, state=None, final_state=None,
               lengths=None, out=None, stream=None):
    """Short causal convolution: y_t = act(bias + sum_k weight[:, k] *
    x_(t-K+1+k)) per channel, with ``state`` (or zeros) before the first
    position.  x: (N, C, L); weight: (C, K) float32, K = 1..4; bias: (C,)
    float32; state: (N, C, K-1), the inputs before x; lengths: (N,) int32, outputs behind
    them are zero; final_state (optional, same shape as state): overwritten
    with the state behind the last position.  Returns y (``out`` if given)."""
    N, C, L = _dims(x, 3, "x")
    K = _dims(weight, 2, "weight")[1]
    c = _Call(x, "x", stream)
    f32, i32 = c.torch.float32, c.torch.int32
    a = ShortConvArgs(N, C, L, K, c.code, bool(silu))
    a.x, a.x_stride_n, a.x_stride_c = c.rows(x, "x", x.shape), x.stride(0), x.stride(1)
    a.weight = c.whole(weight, "weight", (C, K), f32)
    a.bias = c.whole(bias, "bias", (C,), f32)
    a.state = c.whole(state, "state", (N, C, K - 1))
    a.final_state = c.whole(final_state, "final_state", (N, C, K - 1))
    a.lengths = c.whole(lengths, "lengths", (N,), i32)
    y = c.out(out, "out", (N, C, L))
    a.y = y.data_ptr()
    c.run("spconv_short_conv", a)
    return y


def short_conv_backward(dy, x, weight, bias=None, *, silu: bool = True, state=None,
                        dfinal_state=None, lengths=None, stream=None):
    """Gradients of ``short_conv`` called with the same arguments, from those of
    y (dy) and, optionally, of final_state: (dx, dweight, dbias, dstate), with
    None for dbias without a bias and for dstate without a state."""
    N, C, L = _dims(x, 3, "x")
    K = _dims(weight, 2, "weight")[1]
    c = _Call(x, "x", stream)
    f32, i32 = c.torch.float32, c.torch.int32
    a = ShortConvArgs(N, C, L, K, c.code, bool(silu))
    a.x, a.x_stride_n, a.x_stride_c = c.rows(x, "x", x.shape), x.stride(0), x.stride(1)
    a.dy = c.rows(dy, "dy", x.shape)
    a.dy_stride_n, a.dy_stride_c = dy.stride(0), dy.stride(1)
    a.weight = c.whole(weight, "weight", (C, K), f32)
    a.bias = c.whole(bias, "bias", (C,), f32)
    a.state = c.whole(state, "state", (N, C, K - 1))
    a.dfinal_state = c.whole(dfinal_state, "dfinal_state", (N, C, K - 1))
    a.lengths = c.whole(lengths, "lengths", (N,), i32)
    dx, dw = c.new((N, C, L)), c.new((C, K), f32)
    db = c.new((C,), f32) if bias is not None else None
    ds = c.new((N, C, K - 1)) if state is not None else None
    a.dx, a.dweight = dx.data_ptr(), dw.data_ptr()
    a.dbias = db.data_ptr() if db is not None else None
    a.dstate = ds.data_ptr() if ds is not None else None
    keep = c.workspace(a, "spconv_short_conv_backward_workspace")
    c.run("spconv_short_conv_backward", a)
    del keep
    return dx, dw, db, ds


def short_conv_step(x, state, weight, bias=None, *, silu: bool = True, slots=None, out=None,
                    stream=None):
    """One position of each of N requests: x (N, C) -> y (N, C), and ``state``
    (num_slots, C, K-1) moved on in place.  Request n uses state slots[n] ((N,)
    int32; None: number n); one whose slot is outside gets zeros and changes
    nothing."""
    N, C = _dims(x, 2, "x")
    K = _dims(weight, 2, "weight")[1]
    c = _Call(x, "x", stream)
    f32, i32 = c.torch.float32, c.torch.int32
    pool = _dims(state, 3, "state")[0]
    a = ShortConvArgs(N, C, 1, K, c.code, bool(silu), pool)
    a.x, a.x_stride_n, a.x_stride_c = c.rows(x, "x", x.shape), x.stride(0), 1
    a.pool = c.whole(state, "state", (pool, C, K - 1))
    a.weight = c.whole(weight, "weight", (C, K), f32)
    a.bias = c.whole(bias, "bias", (C,), f32)
    a.slots = c.whole(slots, "slots", (N,), i32)
    y = c.out(out, "out", (N, C))
    a.y = y.data_ptr()
    c.run("spconv_short_conv_step", a)
    return y


def _scan_args(c, u, delta, A, B, C, D, z, delta_bias, softplus, step, pool):
    """The arguments that the scan's calls share; B and C: (N, S[, L]) or
    (N, groups, S[, L])."""
    f32 = c.torch.float32
    shape = u.shape
    N, ch = shape[0], shape[1]
    S = _dims(A, 2, "A")[1]
    tail = (S,) if step else (S, shape[2])
    G = B.shape[1] if getattr(B, "dim", lambda: -1)() == 2 + len(tail) else 1
    if G < 1 or ch % G:
        _fail("the groups of B and C must divide the channels")
    a = ScanArgs(N, ch, 1 if step else shape[2], S, G, c.code, bool(softplus), pool)
    for t, name in ((u, "u"), (delta, "delta"), (z, "z")):
        if t is not None:
            setattr(a, name, c.rows(t, name, shape))
            setattr(a, name + "_stride_n", t.stride(0))
            setattr(a, name + "_stride_c", 1 if step else t.stride(1))
    for t, name, low in ((B, "B", "b"), (C, "C", "c")):
        grouped = getattr(t, "dim", lambda: -1)() == 2 + len(tail)
        p = c.rows(t, name, (N, G) + tail if grouped else (N,) + tail)
        setattr(a, name, p)
        setattr(a, low + "_stride_n", t.stride(0))
        setattr(a, low + "_stride_g", t.stride(1) if grouped else 0)
        setattr(a, low + "_stride_s", 1 if step else t.stride(-2))
    a.A = c.whole(A, "A", (ch, S), f32)
    a.D = c.whole(D, "D", (ch,), f32)
    a.delta_bias = c.whole(delta_bias, "delta_bias", (ch,), f32)
    return a, S


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
    shape = _dims(u, 3, "u")
    c = _Call(u, "u", stream)
    f32, i32 = c.torch.float32, c.torch.int32
    a, S = _scan_args(c, u, delta, A, B, C, D, z, delta_bias, softplus, False, 0)
    states = (shape[0], shape[1], S)
    a.state = c.whole(state, "state", states, f32)
    a.final_state = c.whole(final_state, "final_state", states, f32)
    a.lengths = c.whole(lengths, "lengths", (shape[0],), i32)
    y = c.out(out, "out", shape)
    a.y = y.data_ptr()
    keep = c.workspace(a, "spconv_scan_workspace")
    c.run("spconv_scan", a)
    del keep
    return y


def scan_backward(dy, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, softplus: bool = True,
                  state=None, dfinal_state=None, lengths=None, stream=None) -> dict:
    """Gradients of ``scan`` called with the same arguments, from those of y (dy)
    and, optionally, of final_state: a dict of du, ddelta, dA, dB, dC, dD, dz,
    ddelta_bias and dstate, None for an argument that was not given."""
    shape = _dims(u, 3, "u")
    c = _Call(u, "u", stream)
    f32, i32 = c.torch.float32, c.torch.int32
    a, S = _scan_args(c, u, delta, A, B, C, D, z, delta_bias, softplus, False, 0)
    a.dy = c.rows(dy, "dy", shape)
    a.dy_stride_n, a.dy_stride_c = dy.stride(0), dy.stride(1)
    states = (shape[0], shape[1], S)
    a.state = c.whole(state, "state", states, f32)
    a.dfinal_state = c.whole(dfinal_state, "dfinal_state", states, f32)
    a.lengths = c.whole(lengths, "lengths", (shape[0],), i32)
    g = dict(du=c.new(shape), ddelta=c.new(shape), dA=c.new(A.shape, f32), dB=c.new(B.shape),
             dC=c.new(C.shape), dD=c.new(D.shape, f32) if D is not None else None,
             dz=c.new(shape) if z is not None else None,
             ddelta_bias=c.new(delta_bias.shape, f32) if delta_bias is not None else None,
             dstate=c.new(states, f32) if state is not None else None)
    for name, t in g.items():
        if t is not None:
            setattr(a, name, t.data_ptr())
    keep = c.workspace(a, "spconv_scan_backward_workspace")
    c.run("spconv_scan_backward", a)
    del keep
    return g


def scan_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, *, softplus: bool = True,
              slots=None, out=None, stream=None):
    """One position of each of N requests: u, delta, z (N, channels), B and C
    (N, S) or (N, groups, S) -> y (N, channels); ``state`` (num_slots,
    channels, S) float32 is moved on in place.  slots as for
    ``short_conv_step``."""
    N, ch = _dims(u, 2, "u")
    c = _Call(u, "u", stream)
    f32, i32 = c.torch.float32, c.torch.int32
    pool = _dims(state, 3, "state")[0]
    a, S = _scan_args(c, u, delta, A, B, C, D, z, delta_bias, softplus, True, pool)
    a.pool = c.whole(state, "state", (pool, ch, S), f32)
    a.slots = c.whole(slots, "slots", (N,), i32)
    y = c.out(out, "out", (N, ch))
    a.y = y.data_ptr()
    c.run("spconv_scan_step", a)
    return y


def adapter_add(y, x, a, b, index, *, scale=None, out=None, stream=None):
    """Low-rank adapters of many requests beside a shared projection: out[n] =
    y[n] + scale[i] * b[i] (a[i] x[n]) with i = index[n]; out[n] = y[n] where i
    is no adapter (-1).  x: (N, C, P) or, for single tokens, (N, C); y: the
    projection's output, (N, M, P) or (N, M); a: (adapters, R, C) and b:
    (adapters, M, R) of x's type, R = 1..64; index: (N,) int32; scale:
    (adapters,) float32, 1 if None.  out may be y itself.  Returns out."""
    c = _Call(x, "x", stream)
    if x.dim() not in (2, 3):
        _fail("x must have 2 or 3 dimensions")
    N, C = x.shape[0], x.shape[1]
    P = x.shape[2] if x.dim() == 3 else 1
    K, R, _ = _dims(a, 3, "a")
    M = _dims(b, 3, "b")[1]
    f32, i32 = c.torch.float32, c.torch.int32
    g = AdapterArgs(N, P, C, M, R, K, c.code)
    g.x, g.x_stride_n, g.x_stride_c = c.rows(x, "x", x.shape), x.stride(0), x.stride(1)
    g.a = c.whole(a, "a", (K, R, C))
    g.b = c.whole(b, "b", (K, M, R))
    g.index = c.whole(index, "index", (N,), i32)
    g.scale = c.whole(scale, "scale", (K,), f32)
    shape = (N, M, P) if x.dim() == 3 else (N, M)
    g.y = c.whole(y, "y", shape)
    if y is None:
        _fail("y must be given")
    out = c.out(out, "out", shape)
    g.out = out.data_ptr()
    keep = c.workspace(g, "spconv_adapter_workspace")
    c.run("spconv_adapter_add", g)
    del keep
    return out
