"""Thin torch binding of libs5.so: the same entry points as include/s5.h.

Argument marshalling only (for some calls natively, csrc/marshal.cpp).  Every tensor must already be on the GPU with the
documented dtype, contiguous (where a call does not take a pitch between
tokens) and 16-byte aligned; nothing is converted or copied here, and every numeric step runs in the library's kernels.  Complex
arrays are torch.complex64 tensors (interleaved re/im float32, as the C ABI
expects).  Work is queued on the current torch CUDA stream unless ``stream``
is given.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import _native
from ._native import S5_BF16, S5_F32, S5Error, check

_DT = {torch.float32: S5_F32, torch.bfloat16: S5_BF16}
_DT_NAME = {"f32": S5_F32, "bf16": S5_BF16, torch.float32: S5_F32, torch.bfloat16: S5_BF16}


def _ptr(t, name, dtype=None, shape=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream if isinstance(s, torch.cuda.Stream) else int(s)


def s5_workspace_size(B: int, L: int, H: int, P: int) -> int:
    return int(_native.lib().s5_workspace_size(B, L, H, P))


def new_workspace(B: int, L: int, H: int, P: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for s5_forward / s5_forward_varying_dt (the
    caller's allocation, made here with torch for convenience)."""
    n = s5_workspace_size(B, L, H, P)
    if n == 0:
        raise ValueError("invalid sizes for a workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def s5_discretize(lam, log_dt, b_tilde, lambda_bar=None, b_bar=None, stream=None):
    """Zero-order hold; returns (lambda_bar [P] complex64, b_bar [P,H] complex64)."""
    P, H = b_tilde.shape
    if lambda_bar is None:
        lambda_bar = torch.empty(P, dtype=torch.complex64, device=b_tilde.device)
    if b_bar is None:
        b_bar = torch.empty(P, H, dtype=torch.complex64, device=b_tilde.device)
    c64 = torch.complex64
    code = _native.lib().s5_discretize(
        _ptr(lam, "lambda", c64, (P,)), _ptr(log_dt, "log_dt", torch.float32, (P,)),
        _ptr(b_tilde, "b_tilde", c64), P, H, _ptr(lambda_bar, "lambda_bar", c64, (P,)),
        _ptr(b_bar, "b_bar", c64, (P, H)), _stream(stream))
    check("s5_discretize", code)
    return lambda_bar, b_bar


_METHOD = {"zoh": 0, "bilinear": 1}


def s5_discretize_ex(lam, log_dt, b_tilde, method="zoh", clip_re=0.0, dt_scale=1.0, lambda_bar=None,
                     b_bar=None, stream=None):
    """Discretisation with options: method "zoh" or "bilinear", clip_eigs
    threshold clip_re (0 = none; the official value is -1e-4), sampling-rate
    factor dt_scale = old rate / new rate.  Returns (lambda_bar, b_bar)."""
    P, H = b_tilde.shape
    if lambda_bar is None:
        lambda_bar = torch.empty(P, dtype=torch.complex64, device=b_tilde.device)
    if b_bar is None:
        b_bar = torch.empty(P, H, dtype=torch.complex64, device=b_tilde.device)
    c64 = torch.complex64
    code = _native.lib().s5_discretize_ex(
        _ptr(lam, "lambda", c64, (P,)), _ptr(log_dt, "log_dt", torch.float32, (P,)),
        _ptr(b_tilde, "b_tilde", c64), P, H, _METHOD[method], float(clip_re), float(dt_scale),
        _ptr(lambda_bar, "lambda_bar", c64, (P,)), _ptr(b_bar, "b_bar", c64, (P, H)), _stream(stream))
    check("s5_discretize_ex", code)
    return lambda_bar, b_bar


def s5_step(lambda_bar, b_bar, c_tilde, d, x, u, y=None, stream=None):
    """One streaming step: x [B,P] complex64 is updated in place; returns y [B,H]."""
    P, H = b_bar.shape
    Bn = u.shape[0]
    if y is None:
        y = torch.empty(Bn, H, dtype=torch.float32, device=u.device)
    c64 = torch.complex64
    code = _native.lib().s5_step(
        _ptr(lambda_bar, "lambda_bar", c64, (P,)), _ptr(b_bar, "b_bar", c64, (P, H)),
        _ptr(c_tilde, "c_tilde", c64, (H, P)), _ptr(d, "d", torch.float32, (H,)),
        _ptr(x, "x", c64, (Bn, P)), _ptr(u, "u", torch.float32, (Bn, H)),
        _ptr(y, "y", torch.float32, (Bn, H)), Bn, H, P, _stream(stream))
    check("s5_step", code)
    return y


def s5_bidirectional_workspace_size(B, L, H, P, u_dtype=torch.float32, y_dtype=None) -> int:
    y_dtype = u_dtype if y_dtype is None else y_dtype
    return int(_native.lib().s5_bidirectional_workspace_size(B, L, H, P, _DT[u_dtype], _DT[y_dtype]))


def s5_forward_bidirectional(lambda_bar, b_bar, c_tilde2, d, u, y=None, y_dtype=None, proj_dtype="f32",
                             workspace=None, stream=None):
    """Bidirectional S5 layer: c_tilde2 [H,2P] holds the forward modes' C~ in
    columns 0..P-1 and the backward modes' in P..2P-1.  Returns y."""
    P = b_bar.shape[0]
    Bn, L, H = u.shape
    if u.dtype not in _DT:
        raise ValueError("u must be float32 or bfloat16")
    ydt = u.dtype if y_dtype is None else y_dtype
    if isinstance(ydt, str):
        ydt = {"f32": torch.float32, "bf16": torch.bfloat16}[ydt]
    if y is None:
        y = torch.empty(Bn, L, H, dtype=ydt, device=u.device)
    if workspace is None:
        n = s5_bidirectional_workspace_size(Bn, L, H, P, u.dtype, y.dtype)
        if n == 0:
            raise ValueError("invalid sizes for a workspace")
        workspace = torch.zeros(n, dtype=torch.uint8, device=u.device)
    c64 = torch.complex64
    code = _native.lib().s5_forward_bidirectional(
        _ptr(lambda_bar, "lambda_bar", c64, (P,)), _ptr(b_bar, "b_bar", c64, (P, H)),
        _ptr(c_tilde2, "c_tilde2", c64, (H, 2 * P)), _ptr(d, "d", torch.float32, (H,)),
        _ptr(u, "u"), _DT[u.dtype], _ptr(y, "y", None, (Bn, L, H)), _DT[y.dtype], _DT_NAME[proj_dtype],
        Bn, L, H, P, _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    check("s5_forward_bidirectional", code)
    return y


def _fwd_common(u, y, y_dtype, proj_dtype, x0, x_last, workspace, P):
    Bn, L, H = u.shape
    if u.dtype not in _DT:
        raise ValueError("u must be float32 or bfloat16")
    ydt = u.dtype if y_dtype is None else y_dtype
    if isinstance(ydt, str):
        ydt = {"f32": torch.float32, "bf16": torch.bfloat16}[ydt]
    if y is None:
        y = torch.empty(Bn, L, H, dtype=ydt, device=u.device)
    if x_last is True:
        x_last = torch.empty(Bn, P, dtype=torch.complex64, device=u.device)
    if workspace is None:
        workspace = new_workspace(Bn, L, H, P, u.device)
    return Bn, L, H, y, x_last, workspace, _DT_NAME[proj_dtype]


def s5_forward(lambda_bar, b_bar, c_tilde, d, u, y=None, y_dtype=None, proj_dtype="f32",
               x0=None, x_last=None, workspace=None, stream=None):
    """Time-invariant S5 forward.  Returns y, or (y, x_last) when x_last is a
    tensor or True."""
    P = b_bar.shape[0]
    Bn, L, H, y, x_last, ws, pd = _fwd_common(u, y, y_dtype, proj_dtype, x0, x_last, workspace, P)
    c64 = torch.complex64
    code = _native.lib().s5_forward(
        _ptr(lambda_bar, "lambda_bar", c64, (P,)), _ptr(b_bar, "b_bar", c64, (P, H)),
        _ptr(c_tilde, "c_tilde", c64, (H, P)), _ptr(d, "d", torch.float32, (H,)),
        _ptr(u, "u"), _DT[u.dtype], _ptr(y, "y", None, (Bn, L, H)), _DT[y.dtype], pd,
        Bn, L, H, P, _ptr(x0, "x0", c64, (Bn, P), True),
        _ptr(x_last, "x_last", c64, (Bn, P), True), _ptr(ws, "workspace", torch.uint8),
        ws.numel(), _stream(stream))
    check("s5_forward", code)
    return y if x_last is None else (y, x_last)


def s5_forward_varying_dt(lam, log_dt, b_tilde, c_tilde, d, dt_scale, u, y=None, y_dtype=None,
                          proj_dtype="f32", x0=None, x_last=None, workspace=None, stream=None):
    """Irregular-sampling S5 forward (interval dt_scale[b,k]*exp(log_dt[n]))."""
    P = b_tilde.shape[0]
    Bn, L, H, y, x_last, ws, pd = _fwd_common(u, y, y_dtype, proj_dtype, x0, x_last, workspace, P)
    c64 = torch.complex64
    code = _native.lib().s5_forward_varying_dt(
        _ptr(lam, "lambda", c64, (P,)), _ptr(log_dt, "log_dt", torch.float32, (P,)),
        _ptr(b_tilde, "b_tilde", c64, (P, H)), _ptr(c_tilde, "c_tilde", c64, (H, P)),
        _ptr(d, "d", torch.float32, (H,)), _ptr(dt_scale, "dt_scale", torch.float32, (Bn, L)),
        _ptr(u, "u"), _DT[u.dtype], _ptr(y, "y", None, (Bn, L, H)), _DT[y.dtype], pd,
        Bn, L, H, P, _ptr(x0, "x0", c64, (Bn, P), True),
        _ptr(x_last, "x_last", c64, (Bn, P), True), _ptr(ws, "workspace", torch.uint8),
        ws.numel(), _stream(stream))
    check("s5_forward_varying_dt", code)
    return y if x_last is None else (y, x_last)


def s5_forward_noalloc(lambda_bar, b_bar, c_tilde, d, u, y, proj_dtype="f32", x0=None,
                       x_last=None, stream=None):
    """s5_forward for callers that cannot allocate device memory: no workspace,
    and no tensor is created here either (y, and x_last if wanted, are the
    caller's).  The library keeps the carry scratch in a fixed device array of
    S5_NOALLOC_SCRATCH_BYTES; larger problems are rejected.  Calls that overlap
    on the GPU share that array and race, so serialize them."""
    P = b_bar.shape[0]
    Bn, L, H = u.shape
    need = s5_workspace_size(Bn, L, H, P)
    if need > _native.S5_NOALLOC_SCRATCH_BYTES:
        raise S5Error("s5_forward_noalloc", 1,
                      "needs %d bytes of carry scratch, more than the library's fixed %d"
                      % (need, _native.S5_NOALLOC_SCRATCH_BYTES))
    c64 = torch.complex64
    code = _native.lib().s5_forward_noalloc(
        _ptr(lambda_bar, "lambda_bar", c64, (P,)), _ptr(b_bar, "b_bar", c64, (P, H)),
        _ptr(c_tilde, "c_tilde", c64, (H, P)), _ptr(d, "d", torch.float32, (H,)),
        _ptr(u, "u"), _DT[u.dtype], _ptr(y, "y", None, (Bn, L, H)), _DT[y.dtype],
        _DT_NAME[proj_dtype], Bn, L, H, P, _ptr(x0, "x0", c64, (Bn, P), True),
        _ptr(x_last, "x_last", c64, (Bn, P), True), _stream(stream))
    check("s5_forward_noalloc", code)
    return y if x_last is None else (y, x_last)


def s5_sync_status(workspace, stream=None) -> int:
    """Waits for the stream; returns and clears the latched device status."""
    return int(_native.lib().s5_sync_status(_ptr(workspace, "workspace", torch.uint8),
                                            _stream(stream)))


# ---------------------------------------------------------------------------
# Gated delta rule, position rotation, norms of queries and keys.  Here q, k,
# v, o and their gradients may be views with a pitch between tokens (slices of
# a fused projection); a head's values and a token's heads are contiguous.
# Contiguous arrays on the current stream are marshalled natively
# (csrc/marshal.cpp); what that returns None for is taken apart here.
# ---------------------------------------------------------------------------
def _taken(fn, out):
    """Whether the native call did the work; raises its error."""
    if out.__class__ is int:
        check(fn, out)
    return out is not None


def _arr(t, name, dtype, shape):
    """_ptr of a contiguous array that has to be there: one expression where all is well."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, name, dtype, shape)


def _new(t):
    """A contiguous array of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _rows(t, name, dtype=None, shape=None):
    """(address, elements between two tokens) of a [..., H, D] array."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t.data_ptr(), shape[-1] * shape[-2]
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1] * t.shape[-2]
    H, D = t.shape[-2:]
    if (D > 1 and t.stride(-1) != 1) or (H > 1 and t.stride(-2) != D):
        raise ValueError("%s: a token's heads must be contiguous" % name)
    pitch = step = None        # of the innermost token axis, and of the next one out
    for n, st in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        if pitch is None:
            pitch = st
        elif st != step:
            raise ValueError("%s: tokens must be evenly spaced" % name)
        step = n * st
    return t.data_ptr(), H * D if pitch is None else pitch


# current_stream() builds an object: 8 us of a call.  A torch without CUDA lacks it, and has no tensor to need it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Launch:
    """The device and the stream of a call on the given arrays, both current inside it.  The library launches on the
    current device, so that has to be the arrays'.  What is made inside belongs to the call's stream: no other stream's
    work can still be using its memory.  Where that is not the caller's stream, memory that one of the two hands to
    the other (the arrays, and what goes through made()) is not given away before both are done with it."""

    def __init__(self, stream, **arrays):
        self.stream, self.guards, self.home, self.handle = stream, [], None, 0
        self.arrays = {n: t for n, t in arrays.items() if isinstance(t, torch.Tensor) and t.is_cuda}

    def __enter__(self):
        dev = first = None
        for name, t in self.arrays.items():
            if dev is None:
                dev, first = t.device, name
            elif t.device != dev:
                raise ValueError("%s is on %s, %s on %s" % (name, t.device, first, dev))
        if dev is None:                  # no array on a GPU: the checks inside say so
            return self
        side = self.stream
        if side is not None and not isinstance(side, torch.cuda.Stream):
            side = torch.cuda.ExternalStream(int(side), dev) if int(side) else torch.cuda.default_stream(dev)
        if side is not None and side.device != dev:
            raise ValueError("the stream is on %s, the arrays on %s" % (side.device, dev))
        if dev.index != torch.cuda.current_device():
            self._enter(torch.cuda.device(dev))
        if side is None:
            self.handle = _raw_stream(dev.index)
            return self
        self.handle, home = side.cuda_stream, torch.cuda.current_stream(dev)
        if self.handle != home.cuda_stream:
            self.home = home
            for t in self.arrays.values():
                t.record_stream(side)
            self._enter(torch.cuda.stream(side))
        return self

    def _enter(self, guard):
        guard.__enter__()
        self.guards.append(guard)

    def __exit__(self, *error):
        while self.guards:
            self.guards.pop().__exit__(*error)

    def made(self, t):
        if self.home is not None:
            t.record_stream(self.home)
        return t


def _delta_sizes(q, k, v, lead):
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor) or q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError("q, k and v must have %d axes" % (lead + 2))
    if q.dtype not in _DT:
        raise ValueError("q, k and v must be float32 or bfloat16")
    if q.shape[:lead] != v.shape[:lead]:
        raise ValueError("q and v have different tokens")
    return (*q.shape, *v.shape[lead:])


def s5_delta_saved_size(B: int, L: int, Hv: int, Dk: int, Dv: int) -> int:
    return int(_native.lib().s5_delta_saved_size(B, L, Hv, Dk, Dv))


def s5_delta_workspace_size(B: int, L: int, Hv: int, Dk: int, Dv: int, backward: bool = False) -> int:
    return int(_native.lib().s5_delta_workspace_size(B, L, Hv, Dk, Dv, int(backward)))


def _buffer(n, what, device):
    if n == 0:
        raise S5Error(what, 2, "head sizes are multiples of 4 up to 256")
    return torch.empty(n, dtype=torch.uint8, device=device)


def new_delta_saved(q, v) -> torch.Tensor:
    """The buffer that s5_delta_forward fills for s5_delta_backward."""
    B, L, _, Dk, Hv, Dv = _delta_sizes(q, q, v, 2)
    return _buffer(s5_delta_saved_size(B, L, Hv, Dk, Dv), "new_delta_saved", q.device)


def s5_delta_forward(q, k, v, g, beta, scale=None, s0=None, s_last=None, o=None, saved=None, workspace=None,
                     stream=None):
    """Gated delta rule over whole sequences: q, k [B,L,Hk,Dk], v [B,L,Hv,Dv], g, beta [B,L,Hv] float32,
    from the state s0 [B,Hv,Dk,Dv] float32 (None: zero).  scale defaults to Dk^-0.5.  Returns o, or
    (o, s_last) when s_last is a tensor (it may be s0) or True; with `saved` (new_delta_saved) also what
    s5_delta_backward needs."""
    if stream is None:
        out = _native.marshal().delta_forward(q, k, v, g, beta, scale, s0, s_last, o, saved, workspace)
        if _taken("s5_delta_forward", out):
            return out
    with _Launch(stream, q=q, k=k, v=v, g=g, beta=beta, s0=s0, s_last=s_last, o=o, saved=saved,
                 workspace=workspace) as on:
        B, L, Hk, Dk, Hv, Dv = _delta_sizes(q, k, v, 2)
        f32, dev, dt = torch.float32, q.device, q.dtype
        if o is None:
            o = on.made(_new(v))
        if s_last is True:
            s_last = on.made(torch.empty(B, Hv, Dk, Dv, dtype=f32, device=dev))
        lib = _native.lib()
        if workspace is None:
            workspace = _buffer(lib.s5_delta_workspace_size(B, L, Hv, Dk, Dv, 0), "s5_delta_forward", dev)
        code = lib.s5_delta_forward(
            *_rows(q, "q"), *_rows(k, "k", dt, q.shape), *_rows(v, "v", dt), _DT[dt],
            _ptr(g, "g", f32, (B, L, Hv)), _ptr(beta, "beta", f32, (B, L, Hv)), _ptr(s0, "s0", f32, (B, Hv, Dk, Dv), True),
            Dk ** -0.5 if scale is None else float(scale), B, L, Hk, Hv, Dk, Dv, *_rows(o, "o", dt, v.shape),
            _ptr(s_last, "s_last", f32, (B, Hv, Dk, Dv), True), _ptr(saved, "saved", torch.uint8, None, True),
            0 if saved is None else saved.numel(), _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
            on.handle)
        check("s5_delta_forward", code)
        return o if s_last is None else (o, s_last)


def s5_delta_backward(q, k, v, g, beta, do, saved, scale=None, s0=None, ds_last=None, workspace=None, stream=None):
    """Gradients of sum(do * o) + sum(ds_last * s_last) after s5_delta_forward with the same inputs and `saved`.
    Returns a dict: dq, dk, dv of q's type, dg, dbeta float32, ds0 float32 (None without s0)."""
    if stream is None:
        out = _native.marshal().delta_backward(q, k, v, g, beta, do, saved, scale, s0, ds_last, workspace)
        if _taken("s5_delta_backward", out):
            return out
    with _Launch(stream, q=q, k=k, v=v, g=g, beta=beta, do=do, saved=saved, s0=s0, ds_last=ds_last,
                 workspace=workspace) as on:
        B, L, Hk, Dk, Hv, Dv = _delta_sizes(q, k, v, 2)
        f32, dev, dt = torch.float32, q.device, q.dtype
        e = lambda shape, t: on.made(torch.empty(shape, dtype=t, device=dev))  # noqa: E731
        out = dict(dq=e(q.shape, dt), dk=e(q.shape, dt), dv=e(v.shape, dt), dg=e((B, L, Hv), f32), dbeta=e((B, L, Hv), f32),
                   ds0=None if s0 is None else e((B, Hv, Dk, Dv), f32))
        lib = _native.lib()
        if workspace is None:
            workspace = _buffer(lib.s5_delta_workspace_size(B, L, Hv, Dk, Dv, 1), "s5_delta_backward", dev)
        code = lib.s5_delta_backward(
            *_rows(q, "q"), *_rows(k, "k", dt, q.shape), *_rows(v, "v", dt), _DT[dt],
            _ptr(g, "g", f32, (B, L, Hv)), _ptr(beta, "beta", f32, (B, L, Hv)), _ptr(s0, "s0", f32, (B, Hv, Dk, Dv), True),
            Dk ** -0.5 if scale is None else float(scale), B, L, Hk, Hv, Dk, Dv, *_rows(do, "do", dt, v.shape),
            _ptr(ds_last, "ds_last", f32, (B, Hv, Dk, Dv), True), _ptr(saved, "saved", torch.uint8), saved.numel(),
            out["dq"].data_ptr(), Hk * Dk, out["dk"].data_ptr(), Hk * Dk, out["dv"].data_ptr(), Hv * Dv,
            out["dg"].data_ptr(), out["dbeta"].data_ptr(), None if s0 is None else out["ds0"].data_ptr(),
            _ptr(workspace, "workspace", torch.uint8), workspace.numel(), on.handle)
        check("s5_delta_backward", code)
        return out


def s5_delta_step(q, k, v, g, beta, state, scale=None, o=None, stream=None):
    """One token per sequence: q, k [B,Hk,Dk], v [B,Hv,Dv], g, beta [B,Hv] float32; state [B,Hv,Dk,Dv] float32 is
    updated in place.  Returns o [B,Hv,Dv]."""
    if stream is None:
        out = _native.marshal().delta_step(q, k, v, g, beta, state, scale, o)
        if _taken("s5_delta_step", out):
            return out
    with _Launch(stream, q=q, k=k, v=v, g=g, beta=beta, state=state, o=o) as on:
        B, Hk, Dk, Hv, Dv = _delta_sizes(q, k, v, 1)
        f32, dt = torch.float32, q.dtype
        if o is None:
            o = on.made(_new(v))
        code = _native.lib().s5_delta_step(
            _arr(q, "q", dt, q.shape), _arr(k, "k", dt, q.shape), _arr(v, "v", dt, v.shape), _DT[dt],
            _arr(g, "g", f32, (B, Hv)), _arr(beta, "beta", f32, (B, Hv)), Dk ** -0.5 if scale is None else float(scale),
            B, Hk, Hv, Dk, Dv, _arr(state, "state", f32, (B, Hv, Dk, Dv)), _arr(o, "o", dt, v.shape), on.handle)
        check("s5_delta_step", code)
        return o


def _fault(fn, device):
    with contextlib.nullcontext() if device is None else torch.cuda.device(device):
        code = getattr(_native.lib(), fn)()
    if code < 0:
        raise S5Error(fn, 3, "the flag could not be read")
    return code != 0


def s5_delta_fault(device=None) -> bool:
    """Whether a wait inside s5_delta_forward or s5_delta_backward has run out on the device (the current one) since
    this was last asked: what those calls gave is then not valid.  Waits for the device."""
    return _fault("s5_delta_fault", device)


def s5_rotary_fault(device=None) -> bool:
    """The same for s5_rotary, s5_qk_norm_rotary and s5_qk_norm_rotary_backward."""
    return _fault("s5_rotary_fault", device)


_LAYOUT = {"half": 0, "interleaved": 1}
_NORM = {None: 0, "none": 0, "rms": 1, "l2": 2}


def _rot_args(x, name, positions, freq):
    if not isinstance(x, torch.Tensor) or x.dim() < 3 or x.dtype not in _DT:
        raise ValueError("%s must be a float32 or bfloat16 array [..., H, D]" % name)
    lead = x.shape[:-2]
    T = math.prod(lead)
    if freq is None:
        return T, None, None, 0
    n = freq.shape[0] if isinstance(freq, torch.Tensor) and freq.dim() == 1 else -1
    return T, _arr(positions, "positions", torch.int64, lead), _arr(freq, "freq", torch.float64, (n,)), 2 * n


def s5_rotary(x, positions, freq, layout="half", amplitude=1.0, inverse=False, out=None, stream=None):
    """Rotates the first 2 * len(freq) values of each head of x [..., H, D] by the angles positions [...] (int64) *
    freq (float64, init.rotary_frequencies) and scales them by amplitude; inverse: the transpose (its backward
    pass).  out may be x."""
    if stream is None:
        done = _native.marshal().rotary(x, positions, freq, _LAYOUT[layout], amplitude, int(inverse), out)
        if _taken("s5_rotary", done):
            return done
    with _Launch(stream, x=x, positions=positions, freq=freq, out=out) as on:
        T, pos, fr, rot = _rot_args(x, "x", positions, freq)
        H, D = x.shape[-2:]
        if out is None:
            out = on.made(_new(x))
        code = _native.lib().s5_rotary(*_rows(x, "x", x.dtype, x.shape), _DT[x.dtype], pos, fr, rot, _LAYOUT[layout], float(amplitude),
                                       int(inverse), T, H, D, *_rows(out, "out", x.dtype, x.shape), on.handle)
        check("s5_rotary", code)
        return out


def s5_qk_norm_rotary(q, k, positions, freq, norm="rms", eps=1e-6, q_weight=None, k_weight=None, layout="half",
                      amplitude=1.0, q_out=None, k_out=None, stream=None):
    """Norm of each head ("rms", "l2" or None), its weight [D] float32 (None: ones) and the rotation of s5_rotary, of
    q [..., Hq, D] and k [..., Hk, D] in one launch.  freq None: no rotation.  q_out may be q, k_out may be k."""
    if stream is None:
        out = _native.marshal().qk_norm_rotary(q, k, positions, freq, _NORM[norm], eps, q_weight, k_weight, _LAYOUT[layout],
                                               amplitude, q_out, k_out)
        if _taken("s5_qk_norm_rotary", out):
            return out
    with _Launch(stream, q=q, k=k, positions=positions, freq=freq, q_weight=q_weight, k_weight=k_weight,
                 q_out=q_out, k_out=k_out) as on:
        T, pos, fr, rot = _rot_args(q, "q", positions, freq)
        (Hq, D), Hk, dt, f32 = q.shape[-2:], k.shape[-2], q.dtype, torch.float32
        kshape = torch.Size((*q.shape[:-2], Hk, D))
        if q_out is None:
            q_out = on.made(_new(q))
        if k_out is None:
            k_out = on.made(_new(k))
        code = _native.lib().s5_qk_norm_rotary(
            *_rows(q, "q", dt, q.shape), *_rows(k, "k", dt, kshape), _DT[dt],
            None if q_weight is None else _arr(q_weight, "q_weight", f32, (D,)),
            None if k_weight is None else _arr(k_weight, "k_weight", f32, (D,)), _NORM[norm], float(eps), pos, fr, rot,
            _LAYOUT[layout], float(amplitude), T, Hq, Hk, D, *_rows(q_out, "q_out", dt, q.shape), *_rows(k_out, "k_out", dt, kshape),
            on.handle)
        check("s5_qk_norm_rotary", code)
        return q_out, k_out


def s5_qk_norm_rotary_backward(q, k, dq_out, dk_out, positions, freq, norm="rms", eps=1e-6, q_weight=None,
                               k_weight=None, layout="half", amplitude=1.0, workspace=None, stream=None):
    """Gradients of s5_qk_norm_rotary from those of its outputs.  Returns a dict: dq, dk, and dwq, dwk [D] float32
    (None without the weight)."""
    if stream is None:
        out = _native.marshal().qk_norm_rotary_backward(q, k, dq_out, dk_out, positions, freq, _NORM[norm], eps, q_weight,
                                                        k_weight, _LAYOUT[layout], amplitude, workspace)
        if _taken("s5_qk_norm_rotary_backward", out):
            return out
    with _Launch(stream, q=q, k=k, dq_out=dq_out, dk_out=dk_out, positions=positions, freq=freq,
                 q_weight=q_weight, k_weight=k_weight, workspace=workspace) as on:
        T, pos, fr, rot = _rot_args(q, "q", positions, freq)
        (Hq, D), Hk, dt, f32, dev = q.shape[-2:], k.shape[-2], q.dtype, torch.float32, q.device
        kshape = (*q.shape[:-2], Hk, D)
        lib = _native.lib()
        e = lambda shape, t: on.made(torch.empty(shape, dtype=t, device=dev))  # noqa: E731
        out = dict(dq=e(q.shape, dt), dk=e(kshape, dt), dwq=None if q_weight is None else e((D,), f32),
                   dwk=None if k_weight is None else e((D,), f32))
        if workspace is None and (q_weight is not None or k_weight is not None):
            workspace = _buffer(lib.s5_qk_norm_rotary_workspace_size(D), "s5_qk_norm_rotary_backward", dev)
        code = lib.s5_qk_norm_rotary_backward(
            *_rows(q, "q"), *_rows(k, "k", dt, kshape), _DT[dt], _ptr(q_weight, "q_weight", f32, (D,), True),
            _ptr(k_weight, "k_weight", f32, (D,), True), _NORM[norm], float(eps), pos, fr, rot, _LAYOUT[layout],
            float(amplitude), T, Hq, Hk, D, *_rows(dq_out, "dq_out", dt, q.shape), *_rows(dk_out, "dk_out", dt, kshape),
            out["dq"].data_ptr(), Hq * D, out["dk"].data_ptr(), Hk * D, _ptr(out["dwq"], "dwq", None, None, True),
            _ptr(out["dwk"], "dwk", None, None, True), _ptr(workspace, "workspace", torch.uint8, None, True),
            0 if workspace is None else workspace.numel(), on.handle)
        check("s5_qk_norm_rotary_backward", code)
        return out


# ---------------------------------------------------------------------------
# Gated linear recurrence, short causal convolution, layer norm of a sum.  Rows
# may be views with a pitch between tokens; a token's channels are contiguous.
# reset [B,L] (bool or uint8): the tokens that begin a new sequence.  lengths
# [B] int32: tokens of each row; what lies behind has no effect, and is zero in
# what comes back.
# ---------------------------------------------------------------------------
_MARKS = (torch.bool, torch.uint8)
_ACT = {None: 0, "none": 0, "silu": 1}


def _tokens(t, name, dtype=None, shape=None):
    """(address, elements between two tokens) of a [..., C] array."""
    if isinstance(t, torch.Tensor) and t.dim() >= 1 and not t.is_contiguous():
        return _rows(t.unsqueeze(-2), name, dtype, None if shape is None else torch.Size((*shape[:-1], 1, shape[-1])))
    return _ptr(t, name, dtype, shape), t.shape[-1]


def _maybe_tokens(t, name, dtype, shape):
    return (None, 0) if t is None else _tokens(t, name, dtype, shape)


def _marks(reset, lengths, B, L):
    if reset is not None and reset.dtype not in _MARKS:
        raise ValueError("reset must be bool or uint8")
    return _ptr(reset, "reset", None, (B, L), True), _ptr(lengths, "lengths", torch.int32, (B,), True)


def _channels(x, name, dims):
    if not isinstance(x, torch.Tensor) or x.dim() != dims or x.dtype not in _DT:
        raise ValueError("%s must be a float32 or bfloat16 array of %d axes" % (name, dims))
    return x.shape


def s5_gated_scan_saved_size(B: int, L: int, C: int) -> int:
    return int(_native.lib().s5_gated_scan_saved_size(B, L, C))


def s5_gated_scan_workspace_size(B: int, L: int, C: int) -> int:
    return int(_native.lib().s5_gated_scan_workspace_size(B, L, C))


def _need(n, what):
    if n == 0:
        raise S5Error(what, 2, "sizes that the call does not cover")
    return n


def new_gated_scan_saved(x) -> torch.Tensor:
    """The buffer that s5_gated_scan_forward fills for s5_gated_scan_backward."""
    out = _native.marshal().gated_scan_saved(x)
    if out is not None:
        return out
    B, L, C = _channels(x, "x", 3)
    return torch.empty(_need(s5_gated_scan_saved_size(B, L, C), "new_gated_scan_saved"), dtype=torch.uint8, device=x.device)


def s5_gated_scan_forward(x, gate_a, gate_x, rate, h0=None, h_last=None, reset=None, lengths=None, normalize=True, h=None,
                          saved=None, stream=None):
    """Gated linear recurrence of each channel, h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_x) x with
    a = exp(-rate sigmoid(gate_a)): x, gate_a, gate_x (None: no input gate) [B,L,C], rate [C] float32, from the state h0
    [B,C] float32 (None: zero).  normalize False: without the root.  Returns h, or (h, h_last) when h_last is a tensor
    (it may be h0) or True; with `saved` (new_gated_scan_saved) also what s5_gated_scan_backward needs."""
    if stream is None:
        out = _native.marshal().gated_scan_forward(x, gate_a, gate_x, rate, h0, h_last, reset, lengths, bool(normalize), h, saved)
        if _taken("s5_gated_scan_forward", out):
            return out
    with _Launch(stream, x=x, gate_a=gate_a, gate_x=gate_x, rate=rate, h0=h0, h_last=h_last, reset=reset, lengths=lengths, h=h,
                 saved=saved) as on:
        B, L, C = _channels(x, "x", 3)
        f32, dt = torch.float32, x.dtype
        if h is None:
            h = on.made(_new(x))
        if h_last is True:
            h_last = on.made(torch.empty(B, C, dtype=f32, device=x.device))
        code = _native.lib().s5_gated_scan_forward(
            *_tokens(x, "x"), *_tokens(gate_a, "gate_a", dt, x.shape), *_maybe_tokens(gate_x, "gate_x", dt, x.shape), _DT[dt],
            _ptr(rate, "rate", f32, (C,)), _ptr(h0, "h0", f32, (B, C), True), *_marks(reset, lengths, B, L), int(bool(normalize)),
            B, L, C, *_tokens(h, "h", dt, x.shape), _ptr(h_last, "h_last", f32, (B, C), True),
            _ptr(saved, "saved", torch.uint8, None, True), 0 if saved is None else saved.numel(), on.handle)
        check("s5_gated_scan_forward", code)
        return h if h_last is None else (h, h_last)


def s5_gated_scan_backward(x, gate_a, gate_x, rate, dh, saved, h0=None, dh_last=None, reset=None, lengths=None, normalize=True,
                           workspace=None, stream=None):
    """Gradients of sum(dh * h) + sum(dh_last * h_last) after s5_gated_scan_forward with the same inputs and `saved`.
    Returns a dict: dx, dgate_a, dgate_x (None without gate_x) of x's type, drate and dh0 (None without h0) float32."""
    if stream is None:
        out = _native.marshal().gated_scan_backward(x, gate_a, gate_x, rate, dh, saved, h0, dh_last, reset, lengths,
                                                    bool(normalize), workspace)
        if _taken("s5_gated_scan_backward", out):
            return out
    with _Launch(stream, x=x, gate_a=gate_a, gate_x=gate_x, rate=rate, dh=dh, saved=saved, h0=h0, dh_last=dh_last, reset=reset,
                 lengths=lengths, workspace=workspace) as on:
        B, L, C = _channels(x, "x", 3)
        f32, dt, dev = torch.float32, x.dtype, x.device
        _ptr(h0, "h0", f32, (B, C), True)
        e = lambda shape, t: on.made(torch.empty(shape, dtype=t, device=dev))  # noqa: E731
        out = dict(dx=e(x.shape, dt), dgate_a=e(x.shape, dt), dgate_x=None if gate_x is None else e(x.shape, dt),
                   drate=e((C,), f32), dh0=None if h0 is None else e((B, C), f32))
        if workspace is None:
            workspace = e((_need(s5_gated_scan_workspace_size(B, L, C), "s5_gated_scan_backward"),), torch.uint8)
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        code = _native.lib().s5_gated_scan_backward(
            *_tokens(x, "x"), *_tokens(gate_a, "gate_a", dt, x.shape), *_maybe_tokens(gate_x, "gate_x", dt, x.shape), _DT[dt],
            _ptr(rate, "rate", f32, (C,)), *_marks(reset, lengths, B, L), int(bool(normalize)), B, L, C,
            *_tokens(dh, "dh", dt, x.shape), _ptr(dh_last, "dh_last", f32, (B, C), True), _ptr(saved, "saved", torch.uint8),
            saved.numel(), at(out["dx"]), C, at(out["dgate_a"]), C, at(out["dgate_x"]), 0 if gate_x is None else C,
            at(out["drate"]), at(out["dh0"]), _ptr(workspace, "workspace", torch.uint8), workspace.numel(), on.handle)
        check("s5_gated_scan_backward", code)
        return out


def s5_gated_scan_fault(device=None) -> bool:
    """Whether a wait inside s5_gated_scan_forward or s5_gated_scan_backward has run out on the device (the current one)
    since this was last asked: what those calls gave is then not valid.  Waits for the device."""
    return _fault("s5_gated_scan_fault", device)


def s5_gated_scan_step(x, gate_a, gate_x, rate, state, normalize=True, h=None, stream=None):
    """One token per sequence: x, gate_a, gate_x (or None) [B,C], rate [C] float32; state [B,C] float32 is updated in
    place.  Returns h [B,C] of x's type."""
    if stream is None:
        out = _native.marshal().gated_scan_step(x, gate_a, gate_x, rate, state, bool(normalize), h)
        if _taken("s5_gated_scan_step", out):
            return out
    with _Launch(stream, x=x, gate_a=gate_a, gate_x=gate_x, rate=rate, state=state, h=h) as on:
        B, C = _channels(x, "x", 2)
        f32, dt = torch.float32, x.dtype
        if h is None:
            h = on.made(_new(x))
        code = _native.lib().s5_gated_scan_step(
            _ptr(x, "x"), _ptr(gate_a, "gate_a", dt, x.shape), _ptr(gate_x, "gate_x", dt, x.shape, True), _DT[dt],
            _ptr(rate, "rate", f32, (C,)), int(bool(normalize)), B, C, _ptr(state, "state", f32, (B, C)), _ptr(h, "h", dt, x.shape),
            on.handle)
        check("s5_gated_scan_step", code)
        return h


def s5_short_conv_workspace_size(C: int, K: int) -> int:
    return int(_native.lib().s5_short_conv_workspace_size(C, K))


def _taps(weight, C):
    """Taps of a [C,K] weight."""
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError("weight must have shape (%d, taps)" % C)
    return weight.shape[1]


def s5_short_conv_forward(x, weight, bias=None, activation=None, past=None, past_out=None, reset=None, lengths=None, y=None,
                          stream=None):
    """Causal convolution of each channel of x [B,L,C] along the tokens, weight [C,K] (K from 2 to 8; its last column
    meets the token itself) and bias [C] float32, activation None or "silu".  past [B,K-1,C] of x's type: the inputs
    before the first (None: zeros).  Returns y, or (y, past_out) when past_out is a tensor (it may be past) or True: the
    inputs that the next call takes as its past."""
    if stream is None:
        out = _native.marshal().short_conv_forward(x, weight, bias, _ACT[activation], past, past_out, reset, lengths, y)
        if _taken("s5_short_conv_forward", out):
            return out
    with _Launch(stream, x=x, weight=weight, bias=bias, past=past, past_out=past_out, reset=reset, lengths=lengths, y=y) as on:
        B, L, C = _channels(x, "x", 3)
        K, f32, dt = _taps(weight, C), torch.float32, x.dtype
        if y is None:
            y = on.made(_new(x))
        if past_out is True:
            past_out = on.made(torch.empty(B, max(K - 1, 0), C, dtype=dt, device=x.device))
        code = _native.lib().s5_short_conv_forward(
            *_tokens(x, "x"), _DT[dt], _ptr(weight, "weight", f32), _ptr(bias, "bias", f32, (C,), True), _ACT[activation],
            _ptr(past, "past", dt, (B, K - 1, C), True), *_marks(reset, lengths, B, L), B, L, C, K, *_tokens(y, "y", dt, x.shape),
            _ptr(past_out, "past_out", dt, (B, K - 1, C), True), on.handle)
        check("s5_short_conv_forward", code)
        return y if past_out is None else (y, past_out)


def s5_short_conv_backward(x, weight, dy, bias=None, activation=None, past=None, dpast_out=None, reset=None, lengths=None,
                           workspace=None, stream=None):
    """Gradients of sum(dy * y) + sum(dpast_out * past_out) with s5_short_conv_forward's inputs.  Returns a dict: dx and
    dpast (None without past) of x's type, dweight [C,K] and dbias [C] (None without bias) float32."""
    if stream is None:
        out = _native.marshal().short_conv_backward(x, weight, dy, bias, _ACT[activation], past, dpast_out, reset, lengths, workspace)
        if _taken("s5_short_conv_backward", out):
            return out
    with _Launch(stream, x=x, weight=weight, dy=dy, bias=bias, past=past, dpast_out=dpast_out, reset=reset, lengths=lengths,
                 workspace=workspace) as on:
        B, L, C = _channels(x, "x", 3)
        K, f32, dt, dev = _taps(weight, C), torch.float32, x.dtype, x.device
        e = lambda shape, t: on.made(torch.empty(shape, dtype=t, device=dev))  # noqa: E731
        out = dict(dx=e(x.shape, dt), dweight=e((C, K), f32), dbias=None if bias is None else e((C,), f32),
                   dpast=None if past is None else e((B, max(K - 1, 0), C), dt))
        if workspace is None:
            workspace = e((_need(s5_short_conv_workspace_size(C, K), "s5_short_conv_backward"),), torch.uint8)
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        code = _native.lib().s5_short_conv_backward(
            *_tokens(x, "x"), _DT[dt], _ptr(weight, "weight", f32), _ptr(bias, "bias", f32, (C,), True), _ACT[activation],
            _ptr(past, "past", dt, (B, K - 1, C), True), *_marks(reset, lengths, B, L), B, L, C, K, *_tokens(dy, "dy", dt, x.shape),
            _ptr(dpast_out, "dpast_out", dt, (B, K - 1, C), True), at(out["dx"]), C, at(out["dweight"]), at(out["dbias"]),
            at(out["dpast"]), _ptr(workspace, "workspace", torch.uint8), workspace.numel(), on.handle)
        check("s5_short_conv_backward", code)
        return out


def s5_short_conv_step(x, weight, state, bias=None, activation=None, y=None, stream=None):
    """One token per sequence: x [B,C]; state [B,K-1,C] of x's type, the inputs before it, is moved on in place.
    Returns y [B,C]."""
    if stream is None:
        out = _native.marshal().short_conv_step(x, weight, state, bias, _ACT[activation], y)
        if _taken("s5_short_conv_step", out):
            return out
    with _Launch(stream, x=x, weight=weight, state=state, bias=bias, y=y) as on:
        B, C = _channels(x, "x", 2)
        K, f32, dt = _taps(weight, C), torch.float32, x.dtype
        if y is None:
            y = on.made(_new(x))
        code = _native.lib().s5_short_conv_step(
            _ptr(x, "x"), _DT[dt], _ptr(weight, "weight", f32), _ptr(bias, "bias", f32, (C,), True), _ACT[activation], B, C, K,
            _ptr(state, "state", dt, (B, K - 1, C)), _ptr(y, "y", dt, x.shape), on.handle)
        check("s5_short_conv_step", code)
        return y


def s5_add_layernorm_workspace_size(H: int) -> int:
    return int(_native.lib().s5_add_layernorm_workspace_size(H))


def _norm_rows(x, name):
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.dtype not in _DT:
        raise ValueError("%s must be a float32 or bfloat16 array [..., H]" % name)
    return math.prod(x.shape[:-1]), x.shape[-1]


def new_layernorm_saved(x) -> torch.Tensor:
    """What s5_add_layernorm fills for s5_add_layernorm_backward: mean and 1 / sqrt(var + eps) of each row."""
    out = _native.marshal().layernorm_saved(x)
    return torch.empty(_norm_rows(x, "x")[0], 2, dtype=torch.float32, device=x.device) if out is None else out


def s5_add_layernorm(x, weight=None, bias=None, residual=None, eps=1e-5, y=None, total=None, saved=None, stream=None):
    """Layer norm over the last axis of x [..., H], or of x + residual, with weight and bias [H] float32 (None: ones,
    zeros).  Returns y, with a residual (y, total): total is the sum, rounded to x's type.  y or total may be x or
    residual.  With `saved` (new_layernorm_saved) also what s5_add_layernorm_backward needs."""
    if stream is None:
        out = _native.marshal().add_layernorm(x, weight, bias, residual, eps, y, total, saved)
        if _taken("s5_add_layernorm", out):
            return out
    with _Launch(stream, x=x, weight=weight, bias=bias, residual=residual, y=y, total=total, saved=saved) as on:
        N, H = _norm_rows(x, "x")
        f32, dt = torch.float32, x.dtype
        if total is not None and residual is None:
            raise ValueError("total without a residual")
        if y is None:
            y = on.made(_new(x))
        if total is None and residual is not None:
            total = on.made(_new(x))
        code = _native.lib().s5_add_layernorm(
            *_tokens(x, "x"), *_maybe_tokens(residual, "residual", dt, x.shape), _DT[dt], _ptr(weight, "weight", f32, (H,), True),
            _ptr(bias, "bias", f32, (H,), True), float(eps), N, H, *_tokens(y, "y", dt, x.shape),
            *_maybe_tokens(total, "total", dt, x.shape), _ptr(saved, "saved", f32, (N, 2), True), on.handle)
        check("s5_add_layernorm", code)
        return y if residual is None else (y, total)


def s5_add_layernorm_backward(x, dy, saved, weight=None, bias=None, residual=None, dtotal=None, workspace=None, stream=None):
    """Gradients of sum(dy * y) + sum(dtotal * total) after s5_add_layernorm with the same x, residual and `saved`.
    Returns a dict: dx of x's type, the gradient of x and of the residual alike, dweight and dbias [H] float32 (None
    without the weight, the bias).  The forward's total as x, without a residual, reads an array less; the gradients
    then carry total's rounding."""
    if stream is None:
        out = _native.marshal().add_layernorm_backward(x, dy, saved, weight, bias, residual, dtotal, workspace)
        if _taken("s5_add_layernorm_backward", out):
            return out
    with _Launch(stream, x=x, dy=dy, saved=saved, weight=weight, bias=bias, residual=residual, dtotal=dtotal,
                 workspace=workspace) as on:
        N, H = _norm_rows(x, "x")
        f32, dt, dev = torch.float32, x.dtype, x.device
        _ptr(bias, "bias", f32, (H,), True)
        e = lambda shape, t: on.made(torch.empty(shape, dtype=t, device=dev))  # noqa: E731
        out = dict(dx=e(x.shape, dt), dweight=None if weight is None else e((H,), f32), dbias=None if bias is None else e((H,), f32))
        if workspace is None and not (weight is None and bias is None):
            workspace = e((_need(s5_add_layernorm_workspace_size(H), "s5_add_layernorm_backward"),), torch.uint8)
        at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        code = _native.lib().s5_add_layernorm_backward(
            *_tokens(x, "x"), *_maybe_tokens(residual, "residual", dt, x.shape), *_tokens(dy, "dy", dt, x.shape),
            *_maybe_tokens(dtotal, "dtotal", dt, x.shape), _DT[dt], _ptr(weight, "weight", f32, (H,), True),
            _ptr(saved, "saved", f32, (N, 2)), N, H, at(out["dx"]), H, at(out["dweight"]), at(out["dbias"]),
            _ptr(workspace, "workspace", torch.uint8, None, True), 0 if workspace is None else workspace.numel(), on.handle)
        check("s5_add_layernorm_backward", code)
        return out


__all__ = ["s5_discretize", "s5_discretize_ex", "s5_forward", "s5_forward_varying_dt",
           "s5_forward_bidirectional", "s5_step", "s5_forward_noalloc", "s5_workspace_size",
           "s5_bidirectional_workspace_size", "s5_sync_status", "new_workspace",
           "s5_delta_forward", "s5_delta_backward", "s5_delta_step", "s5_delta_saved_size",
           "s5_delta_workspace_size", "s5_delta_fault", "new_delta_saved", "s5_rotary", "s5_qk_norm_rotary",
           "s5_qk_norm_rotary_backward", "s5_rotary_fault", "s5_gated_scan_forward", "s5_gated_scan_backward",
           "s5_gated_scan_step", "s5_gated_scan_fault", "s5_gated_scan_saved_size", "s5_gated_scan_workspace_size", "new_gated_scan_saved",
           "s5_short_conv_forward", "s5_short_conv_backward", "s5_short_conv_step", "s5_short_conv_workspace_size",
           "s5_add_layernorm", "s5_add_layernorm_backward", "s5_add_layernorm_workspace_size", "new_layernorm_saved",
           "S5Error", "S5_F32", "S5_BF16"]
