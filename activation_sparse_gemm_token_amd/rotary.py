"""Rotary positions (include/rtlynx_rope.h): the rotation of the queries and
keys that a block's projections make, its gradient, and the frequency tables.

``rope`` and ``rope_backward`` take strided tensors (slices of a fused Q/K/V
projection included), rotate one or two of them in one launch and need only
the channel stride to be 1.  Argument marshalling only, as in the package's
other bindings; the tables are small host-side vectors in float64.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import _check, _here, _no_graph, _on, _stream, _torch, lib

__all__ = ["rope", "rope_backward", "frequencies", "frequencies_by_parts", "LAYOUTS"]

LAYOUTS = ("half", "interleaved")
_INTERLEAVED, _INVERSE = 0x10, 0x20

_c_i64, _c_vp = ctypes.c_int64, ctypes.c_void_p


class _Tensor(ctypes.Structure):
    """rtl_rope_tensor."""
    _fields_ = [("x", _c_vp), ("y", _c_vp), ("heads", _c_i64)] + [
        (f"{t}_{d}_stride", _c_i64) for t in "xy" for d in ("batch", "token", "head")]


_TENSORS = {n: struct.Struct(f"{9 * n}q") for n in (1, 2)}          # the same as plain words, which pack faster

_SIG = (ctypes.c_int, [_c_vp, ctypes.c_int32, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64,
                       ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), _c_vp, ctypes.c_float, ctypes.c_uint32, _c_vp])


def _fn():
    fn = lib().rtl_rope
    if fn.argtypes is None:
        fn.restype, fn.argtypes = _SIG
    return fn


def frequencies(rot_dim: int, base: float = 10000.0, linear: float = 1.0, ntk: float = 1.0):
    """Radians per position of each of ``rot_dim / 2`` pairs, float64 on the
    host: base^(-2 i / rot_dim).  ``linear`` divides every frequency (positions
    stretched by that factor); ``ntk`` stretches the base so that the slowest
    pair slows by that factor and the fastest not at all."""
    torch = _torch()
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and >= 0")
    if not (base > 0 and linear > 0 and ntk > 0):
        raise ValueError("base, linear and ntk must be positive")
    if ntk != 1.0 and rot_dim > 2:
        base = base * ntk ** (rot_dim / (rot_dim - 2))
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    return torch.exp(i * (-2.0 / max(rot_dim, 1) * math.log(base))) / linear


def frequencies_by_parts(rot_dim: int, factor: float, trained_length: int, base: float = 10000.0,
                         fast_turns: float = 32.0, slow_turns: float = 1.0):
    """Frequencies scaled by parts for contexts ``factor`` times the trained
    one, and the scale that goes with them: pairs that turn more than
    ``fast_turns`` times over ``trained_length`` positions keep their
    frequency, those below ``slow_turns`` are divided by ``factor``, and
    between the two the share moves linearly with the pair's index.
    Returns (float64 host tensor, scale = 0.1 ln(factor) + 1)."""
    torch = _torch()
    if not factor >= 1 or trained_length < 1 or not fast_turns > slow_turns > 0 or not base > 1:
        raise ValueError("need factor >= 1, trained_length >= 1, fast_turns > slow_turns > 0 and base > 1")
    f = frequencies(rot_dim, base)

    def index(turns):                        # pair that turns so often over the trained length
        return rot_dim * math.log(trained_length / (2 * math.pi * turns)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(fast_turns)), 0), min(math.ceil(index(slow_turns)), rot_dim - 1)
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    slow = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - slow) + f / factor * slow, 0.1 * math.log(factor) + 1.0


def _span(t):
    """Bytes [first, past the last) that a tensor's elements lie in."""
    lo = hi = t.data_ptr()
    for n, s in zip(t.shape, t.stride()):
        if n == 0:
            return t.data_ptr(), t.data_ptr()
        if s < 0:
            lo += (n - 1) * s * t.element_size()
        else:
            hi += (n - 1) * s * t.element_size()
    return lo, hi + t.element_size()


def _distinct(t):
    """Whether no two index tuples name one element (by nested extents)."""
    inner = 1
    for s, n in sorted((abs(s), n) for n, s in zip(t.shape, t.stride()) if n > 1):
        if s < inner:
            return False
        inner = s * (n - 1) + inner
    return True


def _same(a, b):
    return a.data_ptr() == b.data_ptr() and a.stride() == b.stride() and a.shape == b.shape


def _meets(off, dims, left):
    """Whether sum(d * s) == off for some integers lo <= d <= hi per (s, lo, hi)
    of ``dims`` (s > 0, largest first).  With nested strides a level leaves few
    candidates; past ``left[0]`` of them in all the answer is yes, unproven."""
    if not dims:
        return off == 0
    s, lo, hi = dims[0]
    low = sum(t * a for t, a, _ in dims[1:])                       # what the smaller strides reach
    high = sum(t * b for t, _, b in dims[1:])
    for d in range(max(lo, -((high - off) // s)), min(hi, (off - low) // s) + 1):
        left[0] -= 1
        if left[0] < 0 or _meets(off - d * s, dims[1:], left):
            return True
    return False


def _apart(a, b):
    """Whether two tensors certainly share no element: disjoint extents, or two
    slices of one tensor (the same strides, any order of the dimensions, any
    number of heads each) no element of which is at the same place."""
    (al, ah), (bl, bh) = _span(a), _span(b)
    if ah <= bl or bh <= al:
        return True
    size = a.element_size()
    off = b.data_ptr() - a.data_ptr()
    if off % size or a.dim() != b.dim():
        return False
    dims = []
    for na, nb, sa, sb in zip(a.shape, b.shape, a.stride(), b.stride()):
        if na > 1 and nb > 1 and sa != sb:
            return False
        s = sa if na > 1 else sb
        if s < 0:
            return False
        if s > 0 and (na > 1 or nb > 1):
            dims.append((s, 1 - nb, na - 1))                       # index in a less index in b
    dims.sort(reverse=True)
    return not _meets(off // size, dims, [1000])


def _check_out(name, t, o):
    if o.dtype != t.dtype:
        raise TypeError(f"out of {name} must be {t.dtype}, got {o.dtype}")
    if o.device != t.device or o.shape != t.shape:
        raise ValueError(f"out of {name} must be on {t.device} with shape {tuple(t.shape)}")
    if (t.shape[-1] > 1 and o.stride(-1) != 1) or not _distinct(o):
        raise ValueError(f"out of {name} must have a channel stride of 1 and no overlapping elements")


def _check_overlap(ins, outs):
    """An output may be its own input and shares no element with any other tensor."""
    for i, o in enumerate(outs):
        for j, (name, t, _) in enumerate(ins):
            if o.numel() and t.numel() and not (i == j and _same(o, t)) and not _apart(o, t):
                raise ValueError(f"an output overlaps {name} (it may be its own input, or share no element with any)")
    if len(outs) == 2 and outs[0].numel() and outs[1].numel() and not _apart(outs[0], outs[1]):
        raise ValueError("the two outputs overlap")


def _rope(x, positions, inv_freq, k, layout, sections, scale, out, k_out, inverse):
    torch = _torch()
    dtype, shape = x.dtype, x.shape
    if dtype is torch.bfloat16:
        flags = 0
    elif dtype is torch.float16:
        flags = 1
    elif dtype is torch.float32:
        flags = 2
    else:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {dtype}")
    if layout == "interleaved":
        flags |= _INTERLEAVED
    elif layout != "half":
        raise ValueError(f"layout must be one of {LAYOUTS}, got {layout!r}")
    if inverse:
        flags |= _INVERSE
    if len(shape) not in (3, 4):
        raise ValueError("x must be [tokens, heads, head_dim] or [batch, tokens, heads, head_dim]")
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    lead, dim = shape[:-2], shape[-1]
    batched = len(lead) == 2
    ins = (("x", x, out),) if k is None else (("x", x, out), ("k", k, k_out))
    outs, words = [], []
    for name, t, o in ins:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        ts, st = t.shape, t.stride()
        if t is not x:
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype} like x, got {t.dtype}")
            if ts[:-2] != lead or ts[-1] != dim:
                raise ValueError(f"{name} must have shape {(*lead, 'heads', dim)}, got {tuple(ts)}")
        if dim > 1 and st[-1] != 1:
            raise ValueError(f"{name}: the channel stride must be 1")
        if o is None:
            o = torch.empty_like(t, memory_format=torch.contiguous_format)
        else:
            _check_out(name, t, o)
        so = o.stride()
        words += (t.data_ptr(), o.data_ptr(), ts[-2])
        words += (*st[:3], *so[:3]) if batched else (0, *st[:2], 0, *so[:2])
        outs.append(o)
    if out is not None or k_out is not None:
        _check_overlap(ins, outs)

    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float64 vector")
    rot = 2 * inv_freq.shape[0]
    if rot > dim:
        raise ValueError(f"inv_freq has {rot // 2} pairs, a head {dim} channels")
    axes, pairs, tail = 1, None, ()
    if sections is not None:
        counts = [int(s) for s in sections]
        if any(s < 0 for s in counts) or sum(counts) != rot // 2:
            raise ValueError(f"sections must be counts that sum to {rot // 2} pairs, got {counts}")
        axes, tail = len(counts), (len(counts),)
        pairs = (ctypes.c_int32 * axes)(*counts)
    if positions.dtype is not torch.int64:
        raise TypeError(f"positions must be int64, got {positions.dtype}")
    ps, pos = positions.shape, positions.stride()
    if ps == lead + tail:
        pos_b, pos_t = pos[:2] if batched else (0, pos[0])
    elif batched and ps == lead[1:] + tail:                       # one row of positions for every sequence
        pos_b, pos_t = 0, pos[0]
    else:
        raise ValueError(f"positions must have shape {(*lead, *tail)}" +
                         (f" or {(*lead[1:], *tail)}" if batched else "") + f", got {tuple(ps)}")
    if axes > 1 and pos[-1] != 1:
        raise ValueError("positions: the axis stride must be 1")
    batch, tokens = lead if batched else (1, lead[0])
    args = (_TENSORS[len(ins)].pack(*words), len(ins), batch, tokens, dim, rot, positions.data_ptr(), pos_b, pos_t,
            axes, pairs, inv_freq.data_ptr(), float(scale), flags)
    stream = _here(x, k, positions, inv_freq)
    if stream is None:
        with _on(x.device, k=k, positions=positions, inv_freq=inv_freq):
            st = _fn()(*args, _stream())
    else:
        st = _fn()(*args, stream)
    _check(st, "rtl_rope")
    return outs[0] if k is None else tuple(outs)


def rope(x, positions, inv_freq, k=None, layout: str = "half", sections=None, scale: float = 1.0, out=None,
         k_out=None):
    """Rotates x (and k) [batch, tokens, heads, head_dim] or [tokens, heads,
    head_dim] (bf16, fp16 or fp32; k may have another number of heads) by
    position * inv_freq.

    ``positions`` int64 [batch, tokens] or [tokens]; with ``sections`` (pairs
    per position axis, at most 4 axes, e.g. frame, row and column) it has a
    last dimension of that many axes.  ``inv_freq`` float64 [rot / 2] on the
    device (``frequencies``); channels past rot are copied.  ``layout``
    "half" pairs channels (i, i + rot / 2), "interleaved" (2i, 2i + 1).
    ``out`` / ``k_out`` may be the input itself.  Returns y, or (y, k's y), without
    an autograd graph (``rope_backward``)."""
    if x.requires_grad or (k is not None and k.requires_grad):
        _no_graph("rotary.rope", "rotary.rope_backward forms it", x, k)
    return _rope(x, positions, inv_freq, k, layout, sections, scale, out, k_out, False)


def rope_backward(dy, positions, inv_freq, k=None, layout: str = "half", sections=None, scale: float = 1.0,
                  out=None, k_out=None):
    """Gradient of ``rope`` with respect to its tensors from the gradients dy
    (and k) of its results; arguments as there."""
    return _rope(dy, positions, inv_freq, k, layout, sections, scale, out, k_out, True)
