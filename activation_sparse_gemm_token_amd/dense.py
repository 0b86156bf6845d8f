"""Dense linear layers with what follows them in one launch, and their gradients
(include/rtlynx_dense.h): output projections into the residual stream, an MLP's first
half, a modulation.  (``layers.LayerPolicy`` calls the plain ``dense_linear`` for the layers that
it leaves dense; those with a bias or an activation of their own go here.)

    z = x w^T + bias,  y = residual + gate * act(z)

Argument marshalling only, as in the package's other bindings.
"""
from __future__ import annotations

import ctypes

from . import _check, _here, _no_graph, _on, _stream, _torch, _workspace, lib

__all__ = ["linear", "linear_backward", "workspace_bytes", "backward_workspace_bytes", "ACTIVATIONS"]

ACTIVATIONS = {None: 0, "gelu": 0x10, "gelu_tanh": 0x20, "silu": 0x30}

_Z_FP32 = 0x200

_i64, _vp, _size, _u32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32
_SIGNATURES = {
    "rtl_linear_workspace_bytes": (_size, [_i64] * 3),
    "rtl_linear": (ctypes.c_int, [_vp] * 4 + [_i64] * 2 + [_vp] + [_i64] * 3 + [_vp] * 3 + [_size, _u32, _vp]),
    "rtl_linear_backward_workspace_bytes": (_size, [_i64] * 4),
    "rtl_linear_backward": (ctypes.c_int, [_vp] * 5 + [_i64] * 5 + [_vp] * 5 + [_size, _u32, _vp]),
}


def _fn(name):
    fn = getattr(lib(), name)
    if fn.argtypes is None:
        fn.restype, fn.argtypes = _SIGNATURES[name]
    return fn


def _run(name, args, stream, t, **tensors):
    """Entry point ``name`` on t's device: on ``stream`` (``_here``'s), or where that is None on the
    device that the named tensors share, made current, and its current stream."""
    if stream is None:
        with _on(t.device, **tensors):
            st = _fn(name)(*args, _stream())
    else:
        st = _fn(name)(*args, stream)
    if st:
        _check(st, name)


def _flags(x, activation):
    torch = _torch()
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, got {activation!r}")
    if x.dtype is torch.bfloat16:
        return ACTIVATIONS[activation]
    if x.dtype is torch.float16:
        return ACTIVATIONS[activation] | 1
    raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")


def _matrix(t, name, dtype, shape):
    """A contiguous device tensor."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _sizes(x, w):
    xs, ws = x.shape, w.shape
    if len(xs) < 1 or len(ws) != 2:
        raise ValueError("x must be [..., K] and w [N, K]")
    n, k = ws
    _matrix(x, "x", x.dtype, (*xs[:-1], k))
    _matrix(w, "w", x.dtype, ws)
    m = 1
    for i in xs[:-1]:
        m *= i
    return m, n, k


def _gate(gate, x, n):
    """(pointer, rows, stride)."""
    if gate is None:
        return None, 1, 0
    if gate.dtype is not x.dtype:
        raise TypeError(f"gate must be {x.dtype}, got {gate.dtype}")
    if not gate.is_cuda:
        raise ValueError("gate must be a device tensor")
    if tuple(gate.shape) != (n,) and not (x.dim() == 3 and tuple(gate.shape) == (x.shape[0], n)):
        raise ValueError(f"gate must have shape {(n,)}" + (f" or {(x.shape[0], n)}" if x.dim() == 3 else "") +
                         f", got {tuple(gate.shape)}")
    if n > 1 and gate.stride(-1) != 1:
        raise ValueError("gate: the channel stride must be 1")
    if gate.dim() == 1 or gate.shape[0] <= 1:
        return gate.data_ptr(), 1, 0
    return gate.data_ptr(), gate.shape[0], gate.stride(0)


def _span(t):
    """Bytes [first, past the last) of a tensor with strides >= 0."""
    if t.numel() == 0:
        return 0, 0
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(out, **tensors):
    lo, hi = _span(out)
    for name, t in tensors.items():
        if t is None:
            continue
        a, b = _span(t)
        if a < hi and lo < b:
            raise ValueError(f"out overlaps {name}")


def workspace_bytes(m: int, n: int, k: int) -> int:
    return int(_fn("rtl_linear_workspace_bytes")(m, n, k))


def linear(x, w, bias=None, activation=None, gate=None, residual=None, out=None, keep: bool = False, workspace=None):
    """y [..., N] = residual + gate * act(x w^T + bias) for x [..., K], w [N, K] (bf16 or
    fp16, K a multiple of 8).

    ``activation`` is None, "gelu", "gelu_tanh" or "silu"; ``bias`` [N]; ``gate`` [N] or, for x
    [batch, tokens, K], [batch, N] (a slice of a modulation row goes as it is); ``residual``
    [..., N].  ``out`` may be the residual itself.  Returns y, or with ``keep`` (y, z), z
    x w^T + bias for ``linear_backward``, fp32 with a gate (whose gradient would carry its
    rounding), else of x's type; without an autograd graph."""
    for t in (x, w, bias, gate, residual):
        if t is not None and t.requires_grad:
            _no_graph("dense.linear", "dense.linear_backward forms it", t)
            break
    flags = _flags(x, activation)
    m, n, k = _sizes(x, w)
    shape = (*x.shape[:-1], n)
    bp = rp = gp = zp = wp = z = None
    rows, stride, size = 1, 0, 0
    if bias is not None:
        _matrix(bias, "bias", x.dtype, (n,))
        bp = bias.data_ptr()
    if residual is not None:
        _matrix(residual, "residual", x.dtype, shape)
        rp = residual.data_ptr()
    if gate is not None:
        gp, rows, stride = _gate(gate, x, n)
    if out is None:
        y = x.new_empty(shape)
    else:
        _matrix(out, "out", x.dtype, shape)
        if out.device != x.device:
            raise ValueError(f"out is on {out.device}, x on {x.device}")
        same = residual is not None and out.data_ptr() == residual.data_ptr()
        _apart(out, x=x, w=w, bias=bias, gate=gate, residual=None if same else residual)
        y = out
    if keep:
        if gate is None:
            z = x.new_empty(shape)
        else:
            z = x.new_empty(shape, dtype=_torch().float32)
            flags |= _Z_FP32
        zp = z.data_ptr()
    if m > 16:                                            # the kernel for few rows needs none
        size = workspace_bytes(m, n, k)
    if workspace is not None or size:
        workspace = _workspace(workspace, size, x.device)
        wp, size = workspace.data_ptr(), workspace.numel()
    _run("rtl_linear", (x.data_ptr(), w.data_ptr(), bp, gp, rows, stride, rp, m, n, k, y.data_ptr(), zp, wp, size, flags),
         _here(x, w, bias, gate, residual), x, w=w, bias=bias, gate=gate, residual=residual)
    return (y, z) if keep else y


def backward_workspace_bytes(m: int, n: int, k: int, gate_rows: int = 1) -> int:
    return int(_fn("rtl_linear_backward_workspace_bytes")(m, n, k, gate_rows))


def linear_backward(dy, x, w, z=None, activation=None, gate=None, need_dx: bool = True, need_dw: bool = True,
                    need_dbias: bool = True, need_dgate: bool = True, workspace=None):
    """Gradients of ``linear`` from dy, its x, w and gate, and the z that it kept: (dx, dw, dbias,
    dgate), None where not asked for (dgate is None without a gate).  The residual's gradient is
    dy.  z, of x's type or fp32, is needed with an activation or a gate's gradient."""
    flags = _flags(x, activation)
    m, n, k = _sizes(x, w)
    shape = (*x.shape[:-1], n)
    _matrix(dy, "dy", x.dtype, shape)
    gp, rows, stride = _gate(gate, x, n)
    need_dgate = need_dgate and gate is not None
    if z is None and (activation is not None or need_dgate):
        raise ValueError("an activation, or a gate's gradient, needs z")
    if z is not None:
        if z.dtype is _torch().float32:
            flags |= _Z_FP32
        _matrix(z, "z", z.dtype if flags & _Z_FP32 else x.dtype, shape)
    dx = x.new_empty(x.shape) if need_dx else None
    dw = x.new_empty((n, k)) if need_dw else None
    dbias = x.new_empty((n,)) if need_dbias else None
    dgate = x.new_empty(gate.shape) if need_dgate else None
    workspace = _workspace(workspace, backward_workspace_bytes(m, n, k, rows), x.device)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _run("rtl_linear_backward", (dy.data_ptr(), x.data_ptr(), w.data_ptr(), ptr(z), gp, rows, stride, m, n, k, ptr(dx), ptr(dw),
                                 ptr(dbias), ptr(dgate), workspace.data_ptr(), workspace.numel(), flags),
         _here(x, dy, w, z, gate), x, dy=dy, w=w, z=z, gate=gate)
    return dx, dw, dbias, dgate
