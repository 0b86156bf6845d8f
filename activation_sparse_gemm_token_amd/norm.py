"""Layer norm of the tokens that a block's projections read, and its gradients
(include/rtlynx_norm.h).

    y = (x - mean) * rstd * (offset + weight) + bias

``weight`` and ``bias`` have one value per channel or one row per sequence (a
block's modulation: ``offset=1`` makes the factor 1 + weight).  Strided tensors
go as they are (slices of a joint sequence, of a modulation row); only the
channel stride must be 1.  Argument marshalling only, as in the package's other
bindings.
"""
from __future__ import annotations

import ctypes

from . import _check, _here, _no_graph, _on, _stream, _torch, _workspace, lib
from .rotary import _apart, _distinct, _same

__all__ = ["layer_norm", "layer_norm_backward", "backward_workspace_bytes", "MAX_CHANNELS"]

MAX_CHANNELS = 32768
_AFFINE_FP32 = 0x10

_i64, _vp, _size, _f, _u32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_uint32
_SIGNATURES = {
    "rtl_layer_norm": (ctypes.c_int, [_vp] + [_i64] * 5 + [_vp, _i64, _vp, _i64, _f, _f, _vp, _i64, _i64, _vp, _vp, _u32, _vp]),
    "rtl_layer_norm_backward_workspace_bytes": (_size, [_i64] * 4),
    "rtl_layer_norm_backward": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i64,
                                               _f, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _size, _u32, _vp]),
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


def _type_flag(torch, t, name):
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return 0
    if dtype is torch.float16:
        return 1
    if dtype is torch.float32:
        return 2
    raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}")


def _layout(t, name):
    """(batch, tokens, batch stride, token stride) of [..., C]; more than three
    dimensions must lie like one row after another."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    shape, stride = t.shape, t.stride()
    if not shape:
        raise ValueError(f"{name} must have a channel dimension")
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the channel stride must be 1")
    if len(shape) == 3:
        return shape[0], shape[1], stride[0], stride[1]
    if len(shape) == 2:
        return 1, shape[0], 0, stride[0]
    if len(shape) == 1:
        return 1, 1, 0, 0
    if not t.is_contiguous():
        raise ValueError(f"{name} with more than three dimensions must be contiguous")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return 1, rows, 0, shape[-1]


def _affine(torch, p, name, x, shape):
    """(pointer, stride between sequences, rows) of weight or bias for x of this shape."""
    c, ps = shape[-1], p.shape
    if p.dtype is not x.dtype and p.dtype is not torch.float32:
        raise TypeError(f"{name} must be {x.dtype} or float32, got {p.dtype}")
    if len(ps) == 1 and ps[0] == c:
        stride, rows = 0, 1
    elif len(ps) == 2 and len(shape) == 3 and ps[0] == shape[0] and ps[1] == c:
        stride, rows = p.stride(0), ps[0]
    else:
        raise ValueError(f"{name} must have shape {(c,)}" + (f" or {(shape[0], c)}" if len(shape) == 3 else "") +
                         f", got {tuple(ps)}")
    if c > 1 and p.stride(-1) != 1:
        raise ValueError(f"{name}: the channel stride must be 1")
    return p.data_ptr(), stride, rows


def _check_out(out, like, **others):
    if out.dtype != like.dtype:
        raise TypeError(f"out must be {like.dtype}, got {out.dtype}")
    if out.device != like.device or out.shape != like.shape:
        raise ValueError(f"out must be on {like.device} with shape {tuple(like.shape)}")
    if not _distinct(out):
        raise ValueError("out must have no overlapping elements")
    for name, t in others.items():
        if t is not None and t.numel() and out.numel() and not (name == "x" and _same(out, t)) and not _apart(out, t):
            raise ValueError(f"out overlaps {name}")


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, offset: float = 0.0, out=None, return_stats: bool = False):
    """Layer norm of x [batch, tokens, C], [tokens, C] or [C] (bf16, fp16 or fp32)
    over its channels.

    ``weight`` [C] or [batch, C] and ``bias`` likewise, of x's type or fp32 (both
    the same); the factor is ``offset + weight``, and 1 without a weight.  ``out``
    may be x itself.  Returns y, or with ``return_stats`` (y, mean, rstd), the
    statistics fp32 of x's shape without the channels, without an autograd graph
    (``layer_norm_backward``)."""
    torch = _torch()
    if x.requires_grad or (weight is not None and weight.requires_grad) or (bias is not None and bias.requires_grad):
        _no_graph("norm.layer_norm", "norm.layer_norm_backward forms it", x, weight, bias)
    flags = _type_flag(torch, x, "x")
    batch, tokens, xb, xt = _layout(x, "x")
    shape = x.shape
    wp = bp = None
    ws = bs = 0
    if weight is not None:
        wp, ws, _ = _affine(torch, weight, "weight", x, shape)
        if weight.dtype is torch.float32:
            flags |= _AFFINE_FP32
    if bias is not None:
        if weight is None:
            raise ValueError("a bias needs a weight")
        if bias.dtype is not weight.dtype:
            raise TypeError(f"bias must be {weight.dtype} like weight, got {bias.dtype}")
        bp, bs, _ = _affine(torch, bias, "bias", x, shape)
    c = shape[-1]
    if out is None:
        y, yb, yt = torch.empty_like(x, memory_format=torch.contiguous_format), tokens * c, c
    else:
        _check_out(out, x, x=x, weight=weight, bias=bias)
        y = out
        _, _, yb, yt = _layout(y, "out")
    mean = rstd = mp = rp = None
    if return_stats:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _run("rtl_layer_norm", (x.data_ptr(), batch, tokens, c, xb, xt, wp, ws, bp, bs, offset, eps, y.data_ptr(), yb, yt, mp, rp,
                            flags), _here(x, weight, bias), x, weight=weight, bias=bias)
    return (y, mean, rstd) if return_stats else y


def backward_workspace_bytes(batch: int, tokens: int, c: int, groups: int) -> int:
    return int(_fn("rtl_layer_norm_backward_workspace_bytes")(batch, tokens, c, groups))


def layer_norm_backward(dy, x, mean, rstd, weight=None, offset: float = 0.0, need_dx: bool = True,
                        need_affine: bool = True, workspace=None):
    """Gradients of ``layer_norm`` from dy, its x and the statistics that it
    returned: (dx, dweight, dbias), None where not asked for.

    dweight and dbias have weight's shape and type, summed over the tokens (and
    the sequences that share a row); without a weight both are None."""
    torch = _torch()
    flags = _type_flag(torch, x, "x")
    shape = x.shape
    if dy.dtype is not x.dtype:
        raise TypeError(f"dy must be {x.dtype} like x, got {dy.dtype}")
    if dy.shape != shape:
        raise ValueError(f"dy must have shape {tuple(shape)}, got {tuple(dy.shape)}")
    batch, tokens, xb, xt = _layout(x, "x")
    _, _, gb, gt = _layout(dy, "dy")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype is not torch.float32 or t.shape != shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape[:-1])}")
    c = shape[-1]
    wp, ws, groups = None, 0, 1
    dw = db = dx = None
    dwp = dbp = dxp = work = None
    size = 0
    if weight is not None:
        wp, ws, groups = _affine(torch, weight, "weight", x, shape)
        if weight.dtype is torch.float32:
            flags |= _AFFINE_FP32
        if need_affine:
            dw = torch.empty_like(weight, memory_format=torch.contiguous_format)
            db = torch.empty_like(dw)
            size = backward_workspace_bytes(batch, tokens, c, groups)
            dwp, dbp = dw.data_ptr(), db.data_ptr()
            if workspace is not None or size:
                workspace = _workspace(workspace, size, x.device)
                work, size = workspace.data_ptr(), workspace.numel()
    if need_dx:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
        dxp = dx.data_ptr()
    _run("rtl_layer_norm_backward",
         (dy.data_ptr(), gb, gt, x.data_ptr(), xb, xt, mean.data_ptr(), rstd.data_ptr(), batch, tokens, c, wp, ws, offset,
          groups, dxp, tokens * c, c, dwp, dbp, work, size, flags),
         _here(x, dy, mean, rstd, weight), x, dy=dy, mean=mean, rstd=rstd, weight=weight)
    return dx, dw, db
