"""The layer operators around the delta rule (include/gdn_layers.h): short causal
convolution, selective state space scan, gated linear recurrence, dropout, RMS norm with
gate or residual sum, and the loss of the model that they make (linear softmax cross entropy).

As in ``binding``: argument checks and marshalling only, every step of the
computation runs in the library's CUDA kernels on the current torch stream, and a
call that cannot run raises (TypeError, ValueError, or GdnError with the library's
status).  The ``dn_*`` functions take caller-owned buffers and carry the C names;
``conv_*``, ``scan_*``, ``recur_*``, ``dropout_*``, ``norm_*`` and ``xent_*`` allocate the results (and workspaces) with
torch and call them.

Token arrays may have any strides as long as the feature axis is contiguous, so
slices and transposed views of a projection go in, and come out (``out=``), without
a copy.  They are float32 or bfloat16, all of one type in a call; parameters (weights,
A, D, biases), scan states and their gradients are float32.

A result must not overlap an input or another result (a single token's new state may be the
old one).  ``conv_forward`` and ``conv_backward``, whose neighbouring tokens would read what
was written over them, refuse an ``out`` that does; the other calls do not look.

Packed sequences: B = 1 and ``cu_seqlens``, int32 offsets on the device, as in
``binding.forward``.  The kernels check the offsets; with ``check_status`` (the
default) a packed call reads the status word afterwards, which waits for the
stream, and raises if they were malformed.  ``xent_*`` does so for its targets.  Other
calls never wait.  The waits inside the recurrence's kernels are bounded; should one run out,
the results behind it are NaN, and ``dn_device_status(ws)`` of the ``ws`` that was passed to the
call, packed or not, says DN_ERR_TIMEOUT.
"""
from __future__ import annotations

import functools
import struct
from typing import Optional

import torch

from . import binding
from .binding import DN_BF16, DN_ERR_INVALID_ARG, DN_F32, GdnError, _check, dn_device_status

EXPORTS = ["dn_conv_workspace_size", "dn_conv_fwd", "dn_conv_bwd", "dn_conv_step", "dn_norm_fwd",
           "dn_norm_workspace_size", "dn_norm_bwd", "dn_scan_workspace_size", "dn_scan_saved_size",
           "dn_scan_fwd", "dn_scan_bwd", "dn_scan_step", "dn_recur_workspace_size", "dn_recur_saved_size",
           "dn_recur_fwd", "dn_recur_bwd", "dn_recur_step", "dn_dropout", "dn_xent_workspace_size", "dn_xent_fwd",
           "dn_xent_bwd"]

_DTYPES = {torch.float32: DN_F32, torch.bfloat16: DN_BF16}
_CONV_SHAPE = struct.Struct("8iq")        # dn_conv_shape
_NORM_SHAPE = struct.Struct("6ifi")       # dn_norm_shape
_SCAN_SHAPE = struct.Struct("8iq")        # dn_scan_shape
_SCAN_IO = struct.Struct("29q")           # dn_scan_io, dn_scan_grads: six views, five pointers
_RECUR_SHAPE = struct.Struct("4ifiq")     # dn_recur_shape
_RECUR_IO = struct.Struct("25q")          # dn_recur_io, dn_recur_grads: five views, five pointers
_DROPOUT_SHAPE = struct.Struct("6id")     # dn_dropout_shape
_XENT_SHAPE = struct.Struct("6iq")        # dn_xent_shape
_VIEW = struct.Struct("4q")               # dn_view

_lib = None


def _L():
    """The library, with this module's entry points declared."""
    global _lib
    if _lib is None:
        import ctypes
        L = binding.lib()
        P, S, I, R = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_char_p   # R: a packed record
        for name, args, res in (
                ("dn_conv_workspace_size", [R, I], S),
                ("dn_conv_fwd", [R, R, P, P, P, R, P, P, S, P], I),
                ("dn_conv_bwd", [R, R, P, P, P, R, P, R, P, P, P, P, S, P], I),
                ("dn_conv_step", [R, R, P, P, P, P, R, P], I),
                ("dn_norm_fwd", [R, R, P, R, R, P, R, R, P], I),
                ("dn_norm_workspace_size", [R], S),
                ("dn_scan_workspace_size", [R, I], S),
                ("dn_scan_saved_size", [R], S),
                ("dn_scan_fwd", [R, R, P, S, P, S, P], I),
                ("dn_scan_bwd", [R, R, R, P, S, P, S, P], I),
                ("dn_scan_step", [R, R, P], I),
                ("dn_recur_workspace_size", [R, I], S),
                ("dn_recur_saved_size", [R], S),
                ("dn_recur_fwd", [R, R, P, S, P, S, P], I),
                ("dn_recur_bwd", [R, R, R, P, S, P, S, P], I),
                ("dn_recur_step", [R, R, P], I),
                ("dn_dropout", [R, R, R, P, R, P], I),
                ("dn_xent_workspace_size", [R, R, R, I], S),
                ("dn_xent_fwd", [R, R, R, R, P, P, P, S, P], I),
                ("dn_xent_bwd", [R, R, R, R, P, R, R, P, P, S, P], I),
                ("dn_norm_bwd", [R, R, P, R, P, R, R, R, R, P, R, R, P, P, S, P], I)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


# ------------------------------------------------------------------ checks

def _tokens(t: torch.Tensor, name: str, shape, dtype) -> torch.Tensor:
    """A token array: CUDA, the call's dtype and shape, contiguous features."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and (t.stride(-1) == 1 or shape[-1] <= 1):
        return t
    if t.dtype is not dtype:
        raise TypeError("%s must be %s like the call's other token arrays, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    raise ValueError("%s: the feature axis must be contiguous (stride 1), got strides %s" % (name, t.stride()))


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype=torch.float32):
    """A dense array (parameter, state) or None."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
        return t
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    raise ValueError("%s must be contiguous" % name)


def _dtype_code(t: torch.Tensor, name: str) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype)) from None


def _result(t: Optional[torch.Tensor], name: str, like: torch.Tensor) -> torch.Tensor:
    """A result like `like`: new and contiguous, or the caller's, whose elements must be distinct."""
    if t is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _tokens(t, name, like.shape, like.dtype)
    if t.get_device() != like.get_device():
        raise ValueError("%s is on %s, the inputs are on %s" % (name, t.device, like.device))
    if any(n > 1 and st == 0 for n, st in zip(t.shape, t.stride())):
        raise ValueError("%s must not repeat memory along an axis (stride 0)" % name)
    return t


def _meet(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors of one type share an element: whether some offset into a minus some offset into b is the
    distance of their first elements.  Axes are tried from the longest stride on, each only over the steps that the
    shorter ones can still make up for; False where that is not decided within 1000 steps (layouts that interleave oddly)."""
    if not a.numel() or not b.numel():
        return False
    span = {}                                # stride -> fewest and most steps of it
    for t, sign in ((a, 1), (b, -1)):
        for n, st in zip(t.shape, t.stride()):
            if n > 1 and st:
                lo, hi = span.get(st, (0, 0))
                span[st] = (lo, hi + n - 1) if sign > 0 else (lo - n + 1, hi)
    axes = sorted(span.items(), reverse=True)
    left = [(0, 0)]                          # least and greatest sum of the axes behind each one
    for st, (lo, hi) in reversed(axes):
        left.append((left[-1][0] + lo * st, left[-1][1] + hi * st))
    left.reverse()
    todo, tries = [(0, (b.data_ptr() - a.data_ptr()) // a.element_size())], 0
    while todo and tries < 1000:
        i, d = todo.pop()
        tries += 1
        if not left[i][0] <= d <= left[i][1]:
            continue
        if i == len(axes):
            return True
        st, (lo, hi) = axes[i]
        lo, hi = max(lo, -((left[i + 1][1] - d) // st)), min(hi, (d - left[i + 1][0]) // st)
        todo.extend((i + 1, d - k * st) for k in range(lo, min(hi, lo + 1000) + 1))
    return False


def _apart(t: Optional[torch.Tensor], name: str, **inputs):
    """Refuses a caller's result (None: none given) that shares memory with an input."""
    if t is not None:
        for n, other in inputs.items():
            if other is not None and _meet(t, other):
                raise ValueError("%s must not overlap %s" % (name, n))


def _same_device(first: torch.Tensor, *rest):
    """All arguments on one device, and that device current (its stream is the one used)."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors on different devices: %s and %s" % (first.device, t.device))
    if torch._C._cuda_getDevice() != dev:
        raise ValueError("%s is not the current CUDA device: call under torch.cuda.device(%d)" % (first.device, dev))


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dims(t: torch.Tensor):
    """B, H, T, d of a token array [B,H,T,d], [B,T,d] (one head) or [R,d] (rows)."""
    s = t.shape
    n = len(s)
    return s if n == 4 else (s[0], 1, s[1], s[2]) if n == 3 else (1, 1, s[0], s[1])


def _view(t: Optional[torch.Tensor]) -> Optional[bytes]:
    """Its dn_view record (None: absent)."""
    if t is None:
        return None
    s = t.stride()
    n = len(s)
    if n == 4:
        return _VIEW.pack(t.data_ptr(), s[0], s[1], s[2])
    return _VIEW.pack(t.data_ptr(), s[0], 0, s[1]) if n == 3 else _VIEW.pack(t.data_ptr(), 0, 0, s[0])


def _cu(cu_seqlens, B):
    """(pointer, num_seqs) of packed offsets."""
    if cu_seqlens is None:
        return 0, 0
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise TypeError("cu_seqlens must be a one-dimensional int32 tensor of at least one offset")
    if not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous CUDA tensor")
    if B != 1:
        raise ValueError("packed sequences need B = 1, got B = %d" % B)
    return cu_seqlens.data_ptr(), cu_seqlens.numel() - 1


def _buffer(t: torch.Tensor, name: str, like: torch.Tensor) -> torch.Tensor:
    """A caller's workspace or saved buffer: the library writes (reads) its bytes from the first one on."""
    if not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.get_device() != like.get_device():
        raise ValueError("%s is on %s, the inputs are on %s" % (name, t.device, like.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


_STATUS_ONLY = 256       # a workspace of this size holds the status word and nothing else
_status_only = {}


@functools.lru_cache(maxsize=4096)
def _size(what: str, shape: bytes, for_backward: int, device: int) -> int:
    """Bytes of a call's buffer, by its sizes (the library plans anew for each new shape)."""
    f = getattr(_L(), what)
    return int(f(shape, for_backward)) if for_backward >= 0 else int(f(shape))


def _ws(what: str, shape: bytes, for_backward: int, like: torch.Tensor, packed: bool, where: str, waits: bool = False) -> torch.Tensor:
    """Workspace, or (for_backward -1) saved buffer.  Calls that are neither packed nor wait on the device (the recurrence does) leave the
    status word alone: where they need nothing else, all of a device share one buffer that nothing is written to."""
    dev = like.get_device()
    if packed:          # the record holds an address: nothing to remember
        f = getattr(_L(), what)
        n = int(f(shape, for_backward)) if for_backward >= 0 else int(f(shape))
    else:
        n = _size(what, shape, for_backward, dev)
    if n == 0:
        raise GdnError(DN_ERR_INVALID_ARG, where)
    if n == _STATUS_ONLY and not packed and not waits and for_backward >= 0:
        ws = _status_only.get(dev)
        if ws is None:
            ws = _status_only[dev] = torch.zeros(_STATUS_ONLY, dtype=torch.uint8, device=like.device)
        return ws
    return torch.empty(n, dtype=torch.uint8, device=like.device)


# ------------------------------------------------------------------ convolution

def conv_shape(x: torch.Tensor, width: int, silu: bool = True, cu_seqlens=None) -> bytes:
    """dn_conv_shape record of x [B,H,T,d] or [B,T,C]."""
    B, H, T, d = _dims(x)
    cu, n = _cu(cu_seqlens, B)
    return _CONV_SHAPE.pack(B, H, T, d, width, _dtype_code(x, "x"), 1 if silu else 0, n, cu)


def dn_conv_workspace_size(shape: bytes, for_backward: bool = False) -> int:
    return int(_L().dn_conv_workspace_size(shape, int(for_backward)))


def dn_conv_fwd(shape, x, w, bias, s0, y, sT, ws, stream=None):
    _check(_L().dn_conv_fwd(shape, _view(x), _p(w), _p(bias), _p(s0), _view(y), _p(sT), _p(ws),
                            ws.numel() * ws.element_size(), _stream(stream)), "dn_conv_fwd")


def dn_conv_bwd(shape, x, w, bias, s0, dy, dsT, dx, dw, dbias, ds0, ws, stream=None):
    _check(_L().dn_conv_bwd(shape, _view(x), _p(w), _p(bias), _p(s0), _view(dy), _p(dsT), _view(dx),
                            _p(dw), _p(dbias), _p(ds0), _p(ws), ws.numel() * ws.element_size(),
                            _stream(stream)), "dn_conv_bwd")


def _step_view(t: torch.Tensor) -> bytes:
    """dn_view record of one token a sequence, [n,C] (or a token array [n,H,1,d], [n,1,C])."""
    return _VIEW.pack(t.data_ptr(), t.stride(0), 0, 0) if t.dim() == 2 else _view(t)


def dn_conv_step(shape, x, w, bias, state_in, state_out, y, stream=None):
    _check(_L().dn_conv_step(shape, _step_view(x), _p(w), _p(bias), _p(state_in), _p(state_out), _step_view(y),
                             _stream(stream)), "dn_conv_step")


def _width(w) -> int:
    if w.dim() != 2 or w.shape[1] < 1:
        raise ValueError("w must be [channels, width]")
    return w.shape[1]


def _conv_args(x, w, bias, state, cu_seqlens):
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B,H,T,d] or [B,T,C], got %d axes" % x.dim())
    B, H, T, d = _dims(x)
    _tokens(x, "x", x.shape, x.dtype)
    width = _width(w)
    _dense(w, "w", (H * d, width))
    _dense(bias, "bias", (H * d,))
    n = B if cu_seqlens is None else _cu(cu_seqlens, B)[1]
    _dense(state, "state", (n, width - 1, H * d), x.dtype)
    _same_device(x, w, bias, state, cu_seqlens)
    return n, width


def conv_forward(x, w, bias=None, state=None, cu_seqlens=None, silu=True, out=None, want_state=True, ws=None,
                 check_status=True):
    """Short causal convolution.  x [B,H,T,d] or [B,T,C] (any strides, contiguous features),
    w [C,width] and bias [C] float32 with C = H d, width 2..4; state [N,width-1,C] in x's dtype:
    the inputs before each sequence (None: zero).  Returns (y, final state or None); y is a new
    contiguous tensor of x's shape, or ``out``, which must not overlap x or state."""
    n, width = _conv_args(x, w, bias, state, cu_seqlens)
    y = _result(out, "out", x)
    _apart(out, "out", x=x, state=state)
    sT = torch.empty((n, width - 1, w.shape[0]), dtype=x.dtype, device=x.device) if want_state else None
    shape = conv_shape(x, width, silu, cu_seqlens)
    ws = _ws("dn_conv_workspace_size", shape, 0, x, cu_seqlens is not None, "dn_conv_fwd") if ws is None else _buffer(ws, "ws", x)
    dn_conv_fwd(shape, x, w, bias, state, y, sT, ws)
    if check_status and cu_seqlens is not None:
        _check(dn_device_status(ws), "dn_conv_fwd (device status)")
    return y, sT


def conv_backward(x, w, bias, state, dy, dstate=None, cu_seqlens=None, silu=True, out=None, ws=None, check_status=True):
    """Gradients of <y, dy> + <final state, dstate>: dict dx (x's shape; contiguous, or ``out``, which must
    not overlap x, dy or a state), dw, dbias (None without bias), dstate (of the initial state, None without one)."""
    n, width = _conv_args(x, w, bias, state, cu_seqlens)
    _tokens(dy, "dy", x.shape, x.dtype)
    _dense(dstate, "dstate", (n, width - 1, w.shape[0]), x.dtype)
    _same_device(x, dy, dstate)
    dx = _result(out, "out", x)
    _apart(out, "out", x=x, dy=dy, state=state, dstate=dstate)
    g = dict(dx=dx, dw=torch.empty_like(w), dbias=None if bias is None else torch.empty_like(bias),
             dstate=None if state is None else torch.empty_like(state))
    shape = conv_shape(x, width, silu, cu_seqlens)
    ws = _ws("dn_conv_workspace_size", shape, 1, x, cu_seqlens is not None, "dn_conv_bwd") if ws is None else _buffer(ws, "ws", x)
    dn_conv_bwd(shape, x, w, bias, state, dy, dstate, dx, g["dw"], g["dbias"], g["dstate"], ws)
    if check_status and cu_seqlens is not None:
        _check(dn_device_status(ws), "dn_conv_bwd (device status)")
    return g


def conv_step(x, w, bias=None, state=None, out_state=None, silu=True, out=None):
    """One token per sequence: x [N,C], state [N,width-1,C] (None: zero).  Returns (y, new state); pass
    out_state=state to update the state in place."""
    if x.dim() != 2:
        raise ValueError("x must be [N,C], got %d axes" % x.dim())
    N, C = x.shape
    _tokens(x, "x", x.shape, x.dtype)
    width = _width(w)
    _dense(w, "w", (C, width))
    _dense(bias, "bias", (C,))
    sshape = (N, width - 1, C)
    _dense(state, "state", sshape, x.dtype)
    _same_device(x, w, bias, state, out_state)
    y = _result(out, "out", x)
    if out_state is None:
        out_state = torch.empty(sshape, dtype=x.dtype, device=x.device)
    else:
        _dense(out_state, "out_state", sshape, x.dtype)
    shape = _CONV_SHAPE.pack(N, 1, 1, C, width, _dtype_code(x, "x"), 1 if silu else 0, 0, 0)
    dn_conv_step(shape, x, w, bias, state, out_state, y)
    return y, out_state


# ------------------------------------------------------------------ selective scan

def _flat(t: Optional[torch.Tensor]):
    """[B,T,D], or [n,D] (one token each), as the four numbers of a dn_view."""
    if t is None:
        return 0, 0, 0, 0
    s = t.stride()
    return t.data_ptr(), s[0], 0, s[1] if len(s) == 3 else 0


def _grouped(t: torch.Tensor, tokens: bool = True):
    """B or C likewise (head = group): [B,T,G,N] or [B,T,N], without the T axis for single tokens."""
    s = t.stride()
    tm, s = (s[1], (s[0],) + s[2:]) if tokens else (0, s)
    return t.data_ptr(), s[0], s[1] if len(s) == 3 else 0, tm


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def scan_shape(x: torch.Tensor, Bm: torch.Tensor, dt_softplus: bool = True, cu_seqlens=None) -> bytes:
    """dn_scan_shape record of x [B,T,D] and Bm [B,T,G,N] or [B,T,N] (x [n,D]: single tokens)."""
    xs, bs = x.shape, Bm.shape
    tokens = len(xs) == 3
    cu, n = _cu(cu_seqlens, xs[0])
    G = bs[-2] if len(bs) == (4 if tokens else 3) else 1
    return _SCAN_SHAPE.pack(xs[0], xs[1] if tokens else 1, xs[-1], bs[-1], G, _dtype_code(x, "x"), 1 if dt_softplus else 0, n, cu)


def scan_io(x, dt, A, B, C, D, z, dt_bias, h0, y, hT) -> bytes:
    """dn_scan_io record; x, dt, z, y [B,T,D], B, C [B,T,G,N] or [B,T,N] (x [n,D]: single tokens)."""
    tokens = x.dim() == 3
    return _SCAN_IO.pack(*_flat(x), *_flat(dt), *_grouped(B, tokens), *_grouped(C, tokens), *_flat(z), *_flat(y),
                         A.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(h0), _ptr(hT))


def scan_grads(dy, dx, ddt, dB, dC, dz, dhT, dA, dD, ddt_bias, dh0) -> bytes:
    """dn_scan_grads record."""
    return _SCAN_IO.pack(*_flat(dy), *_flat(dx), *_flat(ddt), *_grouped(dB), *_grouped(dC), *_flat(dz), _ptr(dhT),
                         dA.data_ptr(), _ptr(dD), _ptr(ddt_bias), _ptr(dh0))


def dn_scan_workspace_size(shape: bytes, for_backward: bool = False) -> int:
    return int(_L().dn_scan_workspace_size(shape, int(for_backward)))


def dn_scan_saved_size(shape: bytes) -> int:
    return int(_L().dn_scan_saved_size(shape))


def dn_scan_fwd(shape, io, saved, ws, stream=None):
    _check(_L().dn_scan_fwd(shape, io, _p(saved), 0 if saved is None else saved.numel() * saved.element_size(), _p(ws),
                            ws.numel() * ws.element_size(), _stream(stream)), "dn_scan_fwd")


def dn_scan_bwd(shape, io, grads, saved, ws, stream=None):
    _check(_L().dn_scan_bwd(shape, io, grads, _p(saved), saved.numel() * saved.element_size(), _p(ws),
                            ws.numel() * ws.element_size(), _stream(stream)), "dn_scan_bwd")


def dn_scan_step(shape, io, stream=None):
    _check(_L().dn_scan_step(shape, io, _stream(stream)), "dn_scan_step")


def _scan_args(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, axes):
    """Checks a scan's arguments (axes: of x, 3 or 2); the number of sequences."""
    xs = x.shape
    if len(xs) != axes:
        raise ValueError("x must be %s, got %d axes" % ("[B,T,D]" if axes == 3 else "[n,D]", len(xs)))
    if A.dim() != 2:
        raise ValueError("A must be [D,N]")
    Dc, N = xs[-1], A.shape[1]
    dtype, lead = x.dtype, xs[:-1]
    _dtype_code(x, "x")
    # one group: B and C may come without the group axis
    bs = B.shape
    G = bs[-2] if len(bs) == axes + 1 else 1
    if len(bs) not in (axes, axes + 1) or G < 1 or Dc % G:
        raise ValueError("B must be %s[G,N] (or %s[N]) with G dividing the %d channels" % (("[B,T]", "[B,T]", Dc) if axes == 3 else
                                                                                   ("[n]", "[n]", Dc)))
    _tokens(x, "x", xs, dtype)
    _tokens(dt, "dt", xs, dtype)
    if z is not None:
        _tokens(z, "z", xs, dtype)
    want = lead + (N,) if len(bs) == axes else lead + (G, N)
    _tokens(B, "B", want, dtype)
    _tokens(C, "C", want, dtype)
    _dense(A, "A", (Dc, N))
    _dense(D, "D", (Dc,))
    _dense(dt_bias, "dt_bias", (Dc,))
    n = xs[0] if cu_seqlens is None else _cu(cu_seqlens, xs[0])[1]
    _dense(h0, "h0", (n, Dc, N))
    _same_device(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens)
    return n


def scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, dt_softplus=True, out=None,
                 want_state=True, save=False, ws=None, check_status=True):
    """Selective state space scan.  x, dt, z (gate, optional) [B,T,D]; B, C [B,T,G,N] or [B,T,N];
    A [D,N], D, dt_bias [D] and the initial states h0 [N_seq,D,N] float32; 1 <= N <= 128.  The step is
    softplus(dt + dt_bias) (dt + dt_bias with dt_softplus=False); A <= 0 and steps >= 0 decay.
    Returns (y, hT), or (y, hT, saved) with save=True for scan_backward(saved=saved): the states
    entering every 8th token (16th for N > 32), N / 2 (N / 4) bytes a token and channel."""
    n = _scan_args(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, 3)
    y = _result(out, "out", x)
    hT = torch.empty((n,) + tuple(A.shape), dtype=torch.float32, device=x.device) if want_state else None
    shape = scan_shape(x, B, dt_softplus, cu_seqlens)
    ws = _ws("dn_scan_workspace_size", shape, 0, x, cu_seqlens is not None, "dn_scan_fwd") if ws is None else _buffer(ws, "ws", x)
    saved = _ws("dn_scan_saved_size", shape, -1, x, cu_seqlens is not None, "dn_scan_fwd") if save else None
    dn_scan_fwd(shape, scan_io(x, dt, A, B, C, D, z, dt_bias, h0, y, hT), saved, ws)
    if check_status and cu_seqlens is not None:
        _check(dn_device_status(ws), "dn_scan_fwd (device status)")
    return (y, hT, saved) if save else (y, hT)


def scan_backward(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, dy=None, dhT=None, saved=None, cu_seqlens=None,
                  dt_softplus=True, ws=None, check_status=True):
    """Gradients of <y, dy> + <hT, dhT>, from scan_forward's arguments and ``saved`` buffer.  Returns dict
    dx, ddt, dA, dB, dC, and dD, dz, ddt_bias, dh0 (None for an argument that was not given)."""
    n = _scan_args(x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, 3)
    if dy is None or saved is None:
        raise ValueError("scan_backward needs dy and saved (scan_forward(save=True))")
    _tokens(dy, "dy", x.shape, x.dtype)
    _dense(dhT, "dhT", (n,) + tuple(A.shape))
    _same_device(x, dy, dhT)
    _buffer(saved, "saved", x)
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    g = dict(dx=new(x), ddt=new(x), dA=new(A), dB=new(B), dC=new(C), dD=new(D), dz=new(z), ddt_bias=new(dt_bias), dh0=new(h0))
    shape = scan_shape(x, B, dt_softplus, cu_seqlens)
    ws = _ws("dn_scan_workspace_size", shape, 1, x, cu_seqlens is not None, "dn_scan_bwd") if ws is None else _buffer(ws, "ws", x)
    dn_scan_bwd(shape, scan_io(x, dt, A, B, C, D, z, dt_bias, h0, None, None),
                scan_grads(dy, g["dx"], g["ddt"], g["dB"], g["dC"], g["dz"], dhT, g["dA"], g["dD"], g["ddt_bias"], g["dh0"]), saved, ws)
    if check_status and cu_seqlens is not None:
        _check(dn_device_status(ws), "dn_scan_bwd (device status)")
    return g


def scan_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, out_state=None, dt_softplus=True, out=None):
    """One token per sequence: x, dt, z [n,D], B, C [n,G,N] or [n,N], state [n,D,N] float32 (None: zero).
    Returns (y, new state); pass out_state=state to update the states in place."""
    n = _scan_args(x, dt, A, B, C, D, z, dt_bias, state, None, 2)
    y = _result(out, "out", x)
    sshape = (n,) + A.shape
    if out_state is None:
        out_state = torch.empty(sshape, dtype=torch.float32, device=x.device)
    else:
        _dense(out_state, "out_state", sshape)
        _same_device(x, out_state)
    dn_scan_step(scan_shape(x, B, dt_softplus), scan_io(x, dt, A, B, C, D, z, dt_bias, state, y, out_state))
    return y, out_state


# ------------------------------------------------------------------ gated linear recurrence

def recur_shape(x: torch.Tensor, c: float = 8.0, cu_seqlens=None) -> bytes:
    """dn_recur_shape record of x [B,T,D] (x [n,D]: single tokens)."""
    xs = x.shape
    cu, n = _cu(cu_seqlens, xs[0])
    code = _dtype_code(x, "x")
    try:
        return _RECUR_SHAPE.pack(xs[0], xs[1] if len(xs) == 3 else 1, xs[-1], code, c, n, cu)
    except struct.error:
        raise ValueError("c must be a number and the sizes 32-bit ones, got c = %r, x %s" % (c, tuple(xs))) from None


def recur_io(x, rg, ig, lam, rg_bias, ig_bias, z, h0, y, hT) -> bytes:
    """dn_recur_io record."""
    return _RECUR_IO.pack(*_flat(x), *_flat(rg), *_flat(ig), *_flat(z), *_flat(y), lam.data_ptr(), _ptr(rg_bias), _ptr(ig_bias),
                          _ptr(h0), _ptr(hT))


def recur_grads(dy, dx, drg, dig, dz, dhT, dlam, drg_bias, dig_bias, dh0) -> bytes:
    """dn_recur_grads record."""
    return _RECUR_IO.pack(*_flat(dy), *_flat(dx), *_flat(drg), *_flat(dig), *_flat(dz), _ptr(dhT), dlam.data_ptr(), _ptr(drg_bias),
                          _ptr(dig_bias), _ptr(dh0))


def dn_recur_workspace_size(shape: bytes, for_backward: bool = False) -> int:
    return int(_L().dn_recur_workspace_size(shape, int(for_backward)))


def dn_recur_saved_size(shape: bytes) -> int:
    return int(_L().dn_recur_saved_size(shape))


def dn_recur_fwd(shape, io, saved, ws, stream=None):
    _check(_L().dn_recur_fwd(shape, io, _p(saved), 0 if saved is None else saved.numel() * saved.element_size(), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "dn_recur_fwd")


def dn_recur_bwd(shape, io, grads, saved, ws, stream=None):
    _check(_L().dn_recur_bwd(shape, io, grads, _p(saved), saved.numel() * saved.element_size(), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "dn_recur_bwd")


def dn_recur_step(shape, io, stream=None):
    _check(_L().dn_recur_step(shape, io, _stream(stream)), "dn_recur_step")


def _recur_args(x, rg, ig, lam, rg_bias, ig_bias, z, h0, cu_seqlens, axes):
    """Checks a recurrence's arguments (axes: of x, 3 or 2); the number of sequences."""
    xs = x.shape
    if len(xs) != axes:
        raise ValueError("x must be %s, got %d axes" % ("[B,T,D]" if axes == 3 else "[n,D]", len(xs)))
    _dtype_code(x, "x")
    _tokens(x, "x", xs, x.dtype)
    _tokens(rg, "rg", xs, x.dtype)
    _tokens(ig, "ig", xs, x.dtype)
    if z is not None:
        _tokens(z, "z", xs, x.dtype)
    width = (xs[-1],)
    _dense(lam, "lam", width)
    _dense(rg_bias, "rg_bias", width)
    _dense(ig_bias, "ig_bias", width)
    n = xs[0] if cu_seqlens is None else _cu(cu_seqlens, xs[0])[1]
    _dense(h0, "h0", (n,) + width)
    _same_device(x, rg, ig, lam, rg_bias, ig_bias, z, h0, cu_seqlens)
    return n


def recur_forward(x, rg, ig, lam, rg_bias=None, ig_bias=None, z=None, h0=None, c=8.0, cu_seqlens=None, out=None, want_state=True,
                  save=False, ws=None, check_status=True):
    """Gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(ig + ig_bias) x, a = exp(-c softplus(lam)
    sigmoid(rg + rg_bias)), y = h or h silu(z).  x, rg, ig (the gates before their sigmoid) and z [B,T,D]; lam, rg_bias,
    ig_bias [D] and the initial states h0 [N_seq,D] float32.  Returns (y, hT), or (y, hT, saved) with save=True for
    recur_backward(saved=saved): the state entering every 8th token, half a byte a token and channel."""
    n = _recur_args(x, rg, ig, lam, rg_bias, ig_bias, z, h0, cu_seqlens, 3)
    y = _result(out, "out", x)
    hT = torch.empty((n, x.shape[2]), dtype=torch.float32, device=x.device) if want_state else None
    shape = recur_shape(x, c, cu_seqlens)
    packed = cu_seqlens is not None
    ws = _ws("dn_recur_workspace_size", shape, 0, x, packed, "dn_recur_fwd", True) if ws is None else _buffer(ws, "ws", x)
    saved = _ws("dn_recur_saved_size", shape, -1, x, packed, "dn_recur_fwd") if save else None
    dn_recur_fwd(shape, recur_io(x, rg, ig, lam, rg_bias, ig_bias, z, h0, y, hT), saved, ws)
    if check_status and packed:
        _check(dn_device_status(ws), "dn_recur_fwd (device status)")
    return (y, hT, saved) if save else (y, hT)


def recur_backward(x, rg, ig, lam, rg_bias=None, ig_bias=None, z=None, h0=None, dy=None, dhT=None, saved=None, c=8.0, cu_seqlens=None,
                   ws=None, check_status=True):
    """Gradients of <y, dy> + <hT, dhT>, from recur_forward's arguments and ``saved`` buffer.  Returns dict
    dx, drg, dig, dlam, and drg_bias, dig_bias, dz, dh0 (None for an argument that was not given)."""
    n = _recur_args(x, rg, ig, lam, rg_bias, ig_bias, z, h0, cu_seqlens, 3)
    if dy is None or saved is None:
        raise ValueError("recur_backward needs dy and saved (recur_forward(save=True))")
    _tokens(dy, "dy", x.shape, x.dtype)
    _dense(dhT, "dhT", (n, x.shape[2]))
    _same_device(x, dy, dhT)
    _buffer(saved, "saved", x)
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    g = dict(dx=new(x), drg=new(rg), dig=new(ig), dz=new(z), dlam=new(lam), drg_bias=new(rg_bias), dig_bias=new(ig_bias), dh0=new(h0))
    shape = recur_shape(x, c, cu_seqlens)
    packed = cu_seqlens is not None
    ws = _ws("dn_recur_workspace_size", shape, 1, x, packed, "dn_recur_bwd", True) if ws is None else _buffer(ws, "ws", x)
    dn_recur_bwd(shape, recur_io(x, rg, ig, lam, rg_bias, ig_bias, z, h0, None, None),
                 recur_grads(dy, g["dx"], g["drg"], g["dig"], g["dz"], dhT, g["dlam"], g["drg_bias"], g["dig_bias"], g["dh0"]), saved, ws)
    if check_status and packed:
        _check(dn_device_status(ws), "dn_recur_bwd (device status)")
    return g


def recur_step(x, rg, ig, lam, rg_bias=None, ig_bias=None, z=None, state=None, out_state=None, c=8.0, out=None):
    """One token per sequence: x, rg, ig, z [n,D], state [n,D] float32 (None: zero).  Returns (y, new state);
    pass out_state=state to update the states in place."""
    _recur_args(x, rg, ig, lam, rg_bias, ig_bias, z, state, None, 2)
    y = _result(out, "out", x)
    if out_state is None:
        out_state = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    else:
        _dense(out_state, "out_state", x.shape)
        _same_device(x, out_state)
    dn_recur_step(recur_shape(x, c), recur_io(x, rg, ig, lam, rg_bias, ig_bias, z, state, y, out_state))
    return y, out_state


# ------------------------------------------------------------------ dropout

def dn_dropout(x, p, rng, residual, y, stream=None):
    B, H, T, d = _dims(x)
    code = _dtype_code(x, "x")
    try:
        shape = _DROPOUT_SHAPE.pack(B, H, T, d, code, 0, p)
    except struct.error:
        raise ValueError("p must be a number and the sizes 32-bit ones, got p = %r, x %s" % (p, tuple(x.shape))) from None
    _check(_L().dn_dropout(shape, _view(x), _view(residual), _p(rng), _view(y), _stream(stream)), "dn_dropout")


def _dropout(x, p, rng, residual, out, name):
    if x.dim() not in (2, 3, 4):
        raise ValueError("%s must be [R,d], [B,T,d] or [B,H,T,d], got %d axes" % (name, x.dim()))
    _dtype_code(x, name)
    _tokens(x, name, x.shape, x.dtype)
    if residual is not None:
        _tokens(residual, "residual", x.shape, x.dtype)
    if not 0.0 <= p < 1.0:
        raise ValueError("p must be at least 0 and below 1, got %r" % (p,))
    _dense(rng, "rng", (2,), torch.int64)
    _same_device(x, rng, residual)
    y = _result(out, "out", x)
    if x.numel():
        dn_dropout(x, p, rng, residual, y)
    return y


def dropout_forward(x, p, rng, residual=None, out=None):
    """Dropout: y = residual + keep x / (1 - p), keep with probability 1 - p.  x [R,d], [B,T,d] or [B,H,T,d]; rng int64 [2] on the
    device: seed and number of the call (one for each call and step), read by the kernel, so that a captured call draws a new
    mask when they change.  The mask goes by the element's index in x's shape, not by strides, and is not stored.  ``out`` may be x or
    residual itself."""
    return _dropout(x, p, rng, residual, out, "x")


def dropout_backward(dy, p, rng, out=None):
    """Gradient of x: keep dy / (1 - p), with the mask of the forward call's rng.  That of the residual is dy."""
    return _dropout(dy, p, rng, None, out, "dy")


# ------------------------------------------------------------------ norm

def norm_shape(x: torch.Tensor, w: torch.Tensor, eps: float) -> bytes:
    """dn_norm_shape record of x [B,H,T,d], [B,T,d] or [R,d] and w [d] or [H,d]."""
    B, H, T, d = _dims(x)
    return _NORM_SHAPE.pack(B, H, T, d, _dtype_code(x, "x"), 1 if w.dim() == 2 else 0, eps, 0)


def dn_norm_workspace_size(shape: bytes) -> int:
    return int(_L().dn_norm_workspace_size(shape))


def dn_norm_fwd(shape, x, w, z, residual, res_scale, y, sum, stream=None):
    _check(_L().dn_norm_fwd(shape, _view(x), _p(w), _view(z), _view(residual), _p(res_scale), _view(y),
                            _view(sum), _stream(stream)), "dn_norm_fwd")


def dn_norm_bwd(shape, x, w, z, res_scale, sum, dy, dsum, dx, dw, dz, dresidual, dres_scale, ws, stream=None):
    _check(_L().dn_norm_bwd(shape, _view(x), _p(w), _view(z), _p(res_scale), _view(sum), _view(dy),
                            _view(dsum), _view(dx), _p(dw), _view(dz), _view(dresidual), _p(dres_scale),
                            _p(ws), ws.numel() * ws.element_size(), _stream(stream)), "dn_norm_bwd")


def _norm_args(x, w, res_scale, **more):
    if x.dim() not in (2, 3, 4):
        raise ValueError("x must be [R,d], [B,T,d] or [B,H,T,d], got %d axes" % x.dim())
    _tokens(x, "x", x.shape, x.dtype)
    _, H, _, d = _dims(x)
    _dense(w, "w", (H, d) if w.dim() == 2 else (d,))
    _dense(res_scale, "res_scale", (d,))
    for name, t in more.items():
        if t is not None:
            _tokens(t, name, x.shape, x.dtype)
    _same_device(x, w, res_scale, *more.values())


def norm_forward(x, w, z=None, residual=None, res_scale=None, eps=1e-6, out=None, out_sum=None):
    """RMS norm over the last axis.  x [R,d], [B,T,d] or [B,H,T,d]; w [d], or [H,d] for a weight per head.
    z: gate, y = rms(r) w silu(z).  residual: r = residual + res_scale x (res_scale [d] float32 or
    None: 1), otherwise r = x.  Returns y, or (y, r) with a residual."""
    _norm_args(x, w, res_scale, z=z, residual=residual)
    if residual is None and (res_scale is not None or out_sum is not None):
        raise ValueError("res_scale and out_sum need a residual")
    y = _result(out, "out", x)
    r = None if residual is None else _result(out_sum, "out_sum", x)
    dn_norm_fwd(norm_shape(x, w, eps), x, w, z, residual, res_scale, y, r)
    return y if residual is None else (y, r)


def norm_backward(x, w, dy, z=None, sum=None, dsum=None, res_scale=None, eps=1e-6, ws=None):
    """Gradients of <y, dy> + <r, dsum>.  Without a residual r = x; with one pass ``sum`` = r as norm_forward
    returned it, and x.  Returns dict dx, dw, dz (with z), dresidual (with sum), dres_scale (with
    res_scale); the others are None.  Without res_scale the gradients of x and of the residual are equal, and
    dx and dresidual are one tensor: clone one before changing either in place."""
    _norm_args(x, w, res_scale, dy=dy, z=z, sum=sum, dsum=dsum)
    if sum is None and (res_scale is not None or dsum is not None):
        raise ValueError("res_scale and dsum need sum (the residual sum of the forward pass)")
    new = lambda: torch.empty(x.shape, dtype=x.dtype, device=x.device)  # noqa: E731
    dres = None if sum is None else new()
    # without a scale dx and dresidual are the same gradient: one tensor
    dx = new() if sum is None or res_scale is not None else None
    g = dict(dx=dres if dx is None else dx, dw=torch.empty_like(w), dz=None if z is None else new(), dresidual=dres,
             dres_scale=None if res_scale is None else torch.empty_like(res_scale))
    shape = norm_shape(x, w, eps)
    ws = _ws("dn_norm_workspace_size", shape, -1, x, False, "dn_norm_bwd") if ws is None else _buffer(ws, "ws", x)
    dn_norm_bwd(shape, x, w, z, res_scale, sum, dy, dsum, dx, g["dw"], g["dz"], dres, g["dres_scale"], ws)
    return g


# ------------------------------------------------------------------ linear softmax cross entropy

def xent_shape(x: torch.Tensor, w: torch.Tensor, ignore_index: int = -100) -> bytes:
    """dn_xent_shape record of x [R,K] or [B,T,K] and w [V,K]."""
    B, _, T, K = _dims(x)
    code = _dtype_code(x, "x")
    try:
        return _XENT_SHAPE.pack(B, T, K, w.shape[0], code, 0, ignore_index)
    except struct.error:
        raise ValueError("ignore_index must be a 64-bit integer and the sizes 32-bit ones, got %r, x %s, w %s"
                         % (ignore_index, tuple(x.shape), tuple(w.shape))) from None


def _weight_view(w: torch.Tensor) -> bytes:
    return _VIEW.pack(w.data_ptr(), 0, 0, w.stride(0))


def _token_view(t: torch.Tensor) -> bytes:
    """dn_view record of one value a token, [R] or [B,T]."""
    s = t.stride()
    return _VIEW.pack(t.data_ptr(), s[0] if len(s) == 2 else 0, 0, s[-1])


def dn_xent_workspace_size(shape: bytes, x, w, for_backward: bool = False) -> int:
    return int(_L().dn_xent_workspace_size(shape, _view(x), _weight_view(w), int(for_backward)))


def dn_xent_fwd(shape, x, w, targets, loss, lse, ws, stream=None):
    _check(_L().dn_xent_fwd(shape, _view(x), _weight_view(w), _token_view(targets), _p(loss), _p(lse), _p(ws),
                            ws.numel() * ws.element_size(), _stream(stream)), "dn_xent_fwd")


def dn_xent_bwd(shape, x, w, targets, lse, dloss, dx, dw, ws, stream=None):
    _check(_L().dn_xent_bwd(shape, _view(x), _weight_view(w), _token_view(targets), _p(lse), _token_view(dloss), _view(dx), _p(dw), _p(ws),
                            ws.numel() * ws.element_size(), _stream(stream)), "dn_xent_bwd")


def _per_token(t: torch.Tensor, name: str, shape, dtype) -> torch.Tensor:
    """One value a token, any strides."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    return t


def _xent_args(x, w, targets):
    if x.dim() not in (2, 3):
        raise ValueError("x must be [R,K] or [B,T,K], got %d axes" % x.dim())
    if w.dim() != 2 or w.shape[0] < 1 or w.shape[1] < 1:
        raise ValueError("w must be [vocabulary, K]")
    _dtype_code(x, "x")
    _tokens(x, "x", x.shape, x.dtype)
    _tokens(w, "w", (w.shape[0], x.shape[-1]), x.dtype)
    _per_token(targets, "targets", x.shape[:-1], torch.int64)
    _same_device(x, w, targets)


def _xent_ws(shape, x, w, backward, where):
    n = dn_xent_workspace_size(shape, x, w, backward)
    if n == 0:
        raise GdnError(DN_ERR_INVALID_ARG, where)
    return torch.empty(n, dtype=torch.uint8, device=x.device)


def xent_forward(x, w, targets, ignore_index=-100, ws=None, check_status=True):
    """Softmax cross entropy of the logits x w^T, which are not kept.  x [R,K] or [B,T,K] and w [V,K] of one type, targets int64 of
    x's leading shape.  Returns (loss, lse) of that shape, float32: the loss of each token (0 where its target is ignore_index) and the
    log of the sum of its exponentials, for xent_backward.  A target outside the vocabulary counts as none; with check_status (which
    waits for the stream) it raises."""
    _xent_args(x, w, targets)
    loss = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    shape = xent_shape(x, w, ignore_index)
    ws = _xent_ws(shape, x, w, False, "dn_xent_fwd") if ws is None else _buffer(ws, "ws", x)
    dn_xent_fwd(shape, x, w, targets, loss, lse, ws)
    if check_status:
        _check(dn_device_status(ws), "dn_xent_fwd (device status)")
    return loss, lse


def xent_backward(x, w, targets, lse, dloss, ignore_index=-100, ws=None, check_status=True):
    """Gradients of <loss, dloss>: dict dx, dw, in x's type.  lse as xent_forward returned it, dloss float32 of its shape (any
    strides: one value expanded to all tokens will do).  The logits are made again by pieces of the vocabulary."""
    _xent_args(x, w, targets)
    _dense(lse, "lse", x.shape[:-1])
    _per_token(dloss, "dloss", x.shape[:-1], torch.float32)
    _same_device(x, lse, dloss)
    g = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=x.device), dw=torch.empty(w.shape, dtype=w.dtype, device=w.device))
    shape = xent_shape(x, w, ignore_index)
    ws = _xent_ws(shape, x, w, True, "dn_xent_bwd") if ws is None else _buffer(ws, "ws", x)
    dn_xent_bwd(shape, x, w, targets, lse, dloss, g["dx"], g["dw"], ws)
    if check_status:
        _check(dn_device_status(ws), "dn_xent_bwd (device status)")
    return g
