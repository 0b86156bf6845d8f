"""Attention of the queries, keys and values that a block's projections and
``rotary.rope`` make, and its gradients (include/rtlynx_attention.h).

    o = softmax(scale q k^T) v       over the keys that a query sees

Sequences are rows of a batch, [batch, tokens, heads, head_dim], with all or
(``k_lens``: a cache, a padded batch) some of their keys filled, or lie one
after another, [tokens, heads, head_dim], between ``q_starts``.  Strided heads
go as they are (slices of a fused Q/K/V projection); only the channel stride
must be 1 and the others multiples of 8.  Argument marshalling only, as in the
package's other bindings.
"""
from __future__ import annotations

import ctypes
import math

from . import _check, _here, _no_graph, _on, _stream, _torch, _workspace, lib
from .rotary import _apart, _distinct

__all__ = ["attention", "attention_backward", "workspace_bytes", "backward_workspace_bytes", "MAX_HEAD_DIM"]

MAX_HEAD_DIM = 128
_CAUSAL, _ZERO_REST = 0x10, 0x20

_i64, _vp, _size, _u32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32


class _Tensor(ctypes.Structure):
    """rtl_attn_tensor."""
    _fields_ = [("data", _vp), ("batch_stride", _i64), ("token_stride", _i64), ("head_stride", _i64)]


class _Shape(ctypes.Structure):
    """rtl_attn_shape."""
    _fields_ = [("sequences", _i64), ("tokens_q", _i64), ("tokens_k", _i64), ("heads_q", _i64), ("heads_k", _i64),
                ("head_dim", _i64), ("q_starts", _vp), ("k_starts", _vp), ("k_lens", _vp), ("scale", ctypes.c_float)]


_TP, _SP = ctypes.POINTER(_Tensor), ctypes.POINTER(_Shape)
_SIGNATURES = {
    "rtl_attention_workspace_bytes": (_size, [_SP, _u32]),
    "rtl_attention": (ctypes.c_int, [_TP] * 4 + [_vp, _SP, _vp, _size, _u32, _vp]),
    "rtl_attention_backward_workspace_bytes": (_size, [_SP]),
    "rtl_attention_backward": (ctypes.c_int, [_TP] * 5 + [_vp] + [_TP] * 3 + [_SP, _vp, _size, _u32, _vp]),
}


def _fn(name):
    fn = getattr(lib(), name)
    if fn.argtypes is None:
        fn.restype, fn.argtypes = _SIGNATURES[name]
    return fn


def _run(name, args, t, **tensors):
    stream = _here(t, *tensors.values())
    if stream is None:
        with _on(t.device, **tensors):
            st = _fn(name)(*args, _stream())
    else:
        st = _fn(name)(*args, stream)
    _check(st, name)


def _tensor(t):
    s = t.stride()
    return _Tensor(t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else _Tensor(t.data_ptr(), 0, s[0], s[1])


def _check_tensor(t, name, dtype, dims):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channel stride must be 1")
    if t.numel() and any(s % 8 for s, n in zip(t.stride()[:-1], t.shape) if n > 1):
        raise ValueError(f"{name}: strides must be multiples of 8 elements, got {t.stride()}")


def _even(t):
    """The tensor with strides that the library takes where a dimension of 1 has another."""
    if t.numel() == 0 or any(s % 8 for s in t.stride()[:-1]):
        return t.as_strided(t.shape, [0 if n <= 1 or t.numel() == 0 else s for s, n in zip(t.stride()[:-1], t.shape)] + [1])
    return t


def _index(t, name, n):
    torch = _torch()
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}, got {tuple(t.shape)}")
    return t.data_ptr()


def _shape(q, k, v, scale, q_starts, k_starts, k_lens):
    """Checks the inputs; (shape struct, q, k, v as the library takes them, k_starts)."""
    torch = _torch()
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    packed = q_starts is not None
    if k_starts is not None and not packed:
        raise ValueError("k_starts without q_starts")
    if packed and k_lens is not None:
        raise ValueError("k_lens is for a batch; packed sequences have k_starts")
    dims = 3 if packed else 4
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(t, name, q.dtype, dims)
    if v.shape != k.shape:
        raise ValueError(f"v must have k's shape {tuple(k.shape)}, got {tuple(v.shape)}")
    d = q.shape[-1]
    if k.shape[-1] != d or (not packed and k.shape[0] != q.shape[0]):
        raise ValueError(f"k {tuple(k.shape)} does not match q {tuple(q.shape)}")
    if d < 8 or d > MAX_HEAD_DIM or d % 8:
        raise ValueError(f"head_dim must be a multiple of 8 up to {MAX_HEAD_DIM}, got {d}")
    hq, hk = q.shape[-2], k.shape[-2]
    if (hq % hk if hk else hq):
        raise ValueError(f"{hq} query heads do not share {hk} key heads evenly")
    scale = d ** -0.5 if scale is None else float(scale)
    if not (math.isfinite(scale) and scale >= 0):
        raise ValueError(f"scale must be finite and >= 0, got {scale}")
    s = _Shape(0, q.shape[-3], k.shape[-3], hq, hk, d, None, None, None, scale)
    if packed:
        if q_starts.dim() != 1 or q_starts.shape[0] < 1:
            raise ValueError("q_starts must be a vector of sequences + 1")
        if k_starts is None:
            if k.shape[0] != q.shape[0]:
                raise ValueError(f"k has {k.shape[0]} tokens, q {q.shape[0]}: k_starts is needed")
            k_starts = q_starts
        s.sequences = q_starts.shape[0] - 1
        s.q_starts = _index(q_starts, "q_starts", s.sequences + 1)
        s.k_starts = _index(k_starts, "k_starts", s.sequences + 1)
    else:
        s.sequences = q.shape[0]
        if k_lens is not None:
            s.k_lens = _index(k_lens, "k_lens", s.sequences) if s.sequences else None
    return s, _even(q), _even(k), _even(v), k_starts


def _lse_shape(q):
    return (q.shape[0], q.shape[2], q.shape[1]) if q.dim() == 4 else (q.shape[1], q.shape[0])


def _sizes(q, k, q_starts):
    s = _Shape(q.shape[0] if q_starts is None else q_starts.shape[0] - 1, q.shape[-3], k.shape[-3], q.shape[-2], k.shape[-2],
               q.shape[-1], None, None, None, 1.0)
    if q_starts is not None:
        s.q_starts = s.k_starts = 16                      # only whether there are any counts
    return s


def workspace_bytes(q, k, q_starts=None, causal: bool = False) -> int:
    """Bytes that ``attention`` wants for tensors of these shapes."""
    return int(_fn("rtl_attention_workspace_bytes")(_sizes(q, k, q_starts), _CAUSAL if causal else 0))


def backward_workspace_bytes(q, k, q_starts=None) -> int:
    """Bytes that ``attention_backward`` wants for tensors of these shapes."""
    return int(_fn("rtl_attention_backward_workspace_bytes")(_sizes(q, k, q_starts)))


def attention(q, k, v, causal: bool = False, scale: float = None, q_starts=None, k_starts=None, k_lens=None, out=None,
              return_lse: bool = False, workspace=None):
    """Attention of q [batch, tokens_q, heads_q, head_dim] over k and v [batch, tokens_k,
    heads_k, head_dim] (bf16 or fp16; head_dim a multiple of 8 up to 128; heads_q a
    multiple of heads_k, shared in order).

    ``causal``: query i sees keys j <= i + len_k - len_q.  ``scale`` is head_dim^-1/2 if
    not given.  ``k_lens`` int32 [batch]: only so many keys of each sequence are filled.
    With ``q_starts`` int32 [sequences + 1] the sequences are packed, q [tokens, heads_q,
    head_dim] and k and v likewise (``k_starts``, if theirs differ).  A query that sees no
    key gets zeros.  Rows in no sequence are zeros too, in a given ``out`` (which shares
    no memory with an input) they are left as they were.

    Returns o, or with ``return_lse`` (o, lse), lse fp32 [batch, heads_q, tokens_q] or
    [heads_q, tokens], without an autograd graph (``attention_backward``)."""
    torch = _torch()
    _no_graph("attention.attention", "attention.attention_backward forms it", q, k, v)
    s, q2, k2, v2, k_starts = _shape(q, k, v, scale, q_starts, k_starts, k_lens)
    flags = (0 if q.dtype is torch.bfloat16 else 1) | (_CAUSAL if causal else 0)
    if out is None:
        packed_none = q_starts is not None and s.sequences == 0
        o = (torch.zeros if packed_none else torch.empty)(q.shape, dtype=q.dtype, device=q.device)
        flags |= _ZERO_REST
    else:
        _check_tensor(out, "out", q.dtype, q.dim())
        if out.shape != q.shape or out.device != q.device:
            raise ValueError(f"out must be on {q.device} with shape {tuple(q.shape)}")
        if not _distinct(out):
            raise ValueError("out must have no overlapping elements")
        for name, t in (("q", q), ("k", k), ("v", v), ("q_starts", q_starts), ("k_starts", k_starts), ("k_lens", k_lens)):
            if t is not None and t.numel() and out.numel() and not _apart(out, t):
                raise ValueError(f"out overlaps {name}")
        o = out
    lse = torch.empty(_lse_shape(q), dtype=torch.float32, device=q.device) if return_lse else None
    if lse is not None and s.sequences == 0:
        lse.fill_(-math.inf)
    need = int(_fn("rtl_attention_workspace_bytes")(s, flags))
    if workspace is not None or need:
        workspace = _workspace(workspace, need, q.device)
    args = (_tensor(q2), _tensor(k2), _tensor(v2), _tensor(_even(o)), None if lse is None else lse.data_ptr(), s,
            None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(), flags)
    _run("rtl_attention", args, q, k=k, v=v, q_starts=q_starts, k_starts=k_starts, k_lens=k_lens)
    return (o, lse) if return_lse else o


def attention_backward(d_o, q, k, v, o, lse, causal: bool = False, scale: float = None, q_starts=None, k_starts=None,
                       k_lens=None, workspace=None):
    """Gradients (dq, dk, dv) of ``attention`` from d_o, its inputs, and the o and lse that it
    returned; arguments as there.  bf16 only.  Rows in no sequence, and behind the filled
    keys, are zeros."""
    torch = _torch()
    s, q2, k2, v2, k_starts = _shape(q, k, v, scale, q_starts, k_starts, k_lens)
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"the backward pass is for bfloat16, got {q.dtype}")
    for name, t in (("d_o", d_o), ("o", o)):
        _check_tensor(t, name, q.dtype, q.dim())
        if t.shape != q.shape:
            raise ValueError(f"{name} must have q's shape {tuple(q.shape)}, got {tuple(t.shape)}")
    if lse.dtype is not torch.float32 or tuple(lse.shape) != _lse_shape(q) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {_lse_shape(q)}")
    new = torch.zeros if q_starts is not None and s.sequences == 0 else torch.empty
    dq, dk, dv = (new(t.shape, dtype=q.dtype, device=q.device) for t in (q, k, v))
    workspace = _workspace(workspace, int(_fn("rtl_attention_backward_workspace_bytes")(s)), q.device)
    args = (_tensor(_even(d_o)), _tensor(q2), _tensor(k2), _tensor(v2), _tensor(_even(o)), lse.data_ptr(),
            _tensor(_even(dq)), _tensor(_even(dk)), _tensor(_even(dv)), s, workspace.data_ptr(), workspace.numel(),
            _CAUSAL if causal else 0)
    _run("rtl_attention_backward", args, q, k=k, v=v, d_o=d_o, o=o, lse=lse, q_starts=q_starts, k_starts=k_starts,
         k_lens=k_lens)
    return dq, dk, dv
