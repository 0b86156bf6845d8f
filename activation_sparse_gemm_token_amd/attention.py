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
import struct

from . import _check, _here, _no_graph, _on, _stream, _torch, _workspace, lib
from .rotary import _apart, _distinct

__all__ = ["attention", "attention_backward", "workspace_bytes", "backward_workspace_bytes", "MAX_HEAD_DIM"]

MAX_HEAD_DIM = 128
_CAUSAL, _ZERO_REST = 0x10, 0x20
_TOKEN_STRIDE = 1 << 23                                   # what the header's token strides are below

_i64, _vp, _size, _u32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32


_TENSOR = struct.Struct("4q")                             # rtl_attn_tensor: data, batch, token and head stride
_SHAPE = struct.Struct("9qf4x")                           # rtl_attn_shape: sequences, tokens_q, tokens_k, heads_q, heads_k,
#                                                           head_dim, q_starts, k_starts, k_lens, scale

_SIGNATURES = {
    "rtl_attention_workspace_bytes": (_size, [_vp, _u32]),
    "rtl_attention": (ctypes.c_int, [_vp] * 7 + [_size, _u32, _vp]),
    "rtl_attention_backward_workspace_bytes": (_size, [_vp]),
    "rtl_attention_backward": (ctypes.c_int, [_vp] * 11 + [_size, _u32, _vp]),
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


def _tensor(t, name, dtype, dims):
    """The packed rtl_attn_tensor of a checked tensor."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    s = t.stride()
    if len(s) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(s)}")
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the channel stride must be 1")
    b, tok, h = s[:3] if dims == 4 else (0, *s[:2])
    if (b | tok | h) % 8 or tok >= _TOKEN_STRIDE:         # of a dimension of 1 it does not matter
        used = [0 if n <= 1 or not t.numel() else i for n, i in zip(t.shape, s)]
        b, tok, h = used[:3] if dims == 4 else (0, *used[:2])
        if (b | tok | h) % 8:
            raise ValueError(f"{name}: strides must be multiples of 8 elements, got {s}")
    return _TENSOR.pack(t.data_ptr(), b, tok, h)


def _new(t):
    """The packed rtl_attn_tensor of a contiguous tensor."""
    s = t.shape
    h = s[-1]
    tok = h * s[-2]
    return _TENSOR.pack(t.data_ptr(), tok * s[-3] if len(s) == 4 else 0, tok, h)


def _index(t, name, n):
    torch = _torch()
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}, got {tuple(t.shape)}")
    return t.data_ptr()


def _shape(torch, q, k, v, scale, q_starts, k_starts, k_lens):
    """Checks the inputs: (packed rtl_attn_shape, packed q, k and v, sequences, k_starts)."""
    dtype, qs, ks = q.dtype, q.shape, k.shape
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    packed = q_starts is not None
    if k_starts is not None and not packed:
        raise ValueError("k_starts without q_starts")
    if packed and k_lens is not None:
        raise ValueError("k_lens is for a batch; packed sequences have k_starts")
    dims = 3 if packed else 4
    tensors = _tensor(q, "q", dtype, dims), _tensor(k, "k", dtype, dims), _tensor(v, "v", dtype, dims)
    if v.shape != ks:
        raise ValueError(f"v must have k's shape {tuple(ks)}, got {tuple(v.shape)}")
    hq, d = qs[-2:]
    hk = ks[-2]
    if ks[-1] != d or (not packed and ks[0] != qs[0]):
        raise ValueError(f"k {tuple(ks)} does not match q {tuple(qs)}")
    if d < 8 or d > MAX_HEAD_DIM or d % 8:
        raise ValueError(f"head_dim must be a multiple of 8 up to {MAX_HEAD_DIM}, got {d}")
    if (hq % hk if hk else hq):
        raise ValueError(f"{hq} query heads do not share {hk} key heads evenly")
    scale = d ** -0.5 if scale is None else float(scale)
    if not 0 <= scale < math.inf:
        raise ValueError(f"scale must be finite and >= 0, got {scale}")
    qp = kp = lp = 0
    if packed:
        if q_starts.dim() != 1 or q_starts.shape[0] < 1:
            raise ValueError("q_starts must be a vector of sequences + 1")
        if k_starts is None:
            if ks[0] != qs[0]:
                raise ValueError(f"k has {ks[0]} tokens, q {qs[0]}: k_starts is needed")
            k_starts = q_starts
        n = q_starts.shape[0] - 1
        qp, kp = _index(q_starts, "q_starts", n + 1), _index(k_starts, "k_starts", n + 1)
    else:
        n = qs[0]
        if k_lens is not None:
            lp = _index(k_lens, "k_lens", n)
    return _SHAPE.pack(n, qs[-3], ks[-3], hq, hk, d, qp, kp, lp, scale), tensors, n, k_starts


def _lse_shape(q):
    return (q.shape[0], q.shape[2], q.shape[1]) if q.dim() == 4 else (q.shape[1], q.shape[0])


def _sizes(q, k, q_starts):
    packed = 0 if q_starts is None else 16                # only whether there are any counts
    return _SHAPE.pack(q.shape[0] if q_starts is None else q_starts.shape[0] - 1, q.shape[-3], k.shape[-3], q.shape[-2],
                       k.shape[-2], q.shape[-1], packed, packed, 0, 1.0)


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
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _no_graph("attention.attention", "attention.attention_backward forms it", q, k, v)
    shape, tensors, n, k_starts = _shape(torch, q, k, v, scale, q_starts, k_starts, k_lens)
    flags = (0 if q.dtype is torch.bfloat16 else 1) | (_CAUSAL if causal else 0)
    if out is None:
        o = q.new_empty(q.shape)
        if n == 0:
            o.zero_()
        flags |= _ZERO_REST
        op = _new(o)
    else:
        op = _tensor(out, "out", q.dtype, q.dim())
        if out.shape != q.shape or out.device != q.device:
            raise ValueError(f"out must be on {q.device} with shape {tuple(q.shape)}")
        if not _distinct(out):
            raise ValueError("out must have no overlapping elements")
        for name, t in (("q", q), ("k", k), ("v", v), ("q_starts", q_starts), ("k_starts", k_starts), ("k_lens", k_lens)):
            if t is not None and t.numel() and out.numel() and not _apart(out, t):
                raise ValueError(f"out overlaps {name}")
        o = out
    lse = lp = wp = None
    if return_lse:
        lse = q.new_empty(_lse_shape(q), dtype=torch.float32)
        if n == 0:
            lse.fill_(-math.inf)
        lp = lse.data_ptr()
    size = _fn("rtl_attention_workspace_bytes")(shape, flags)
    if workspace is not None or size:
        workspace = _workspace(workspace, size, q.device)
        wp, size = workspace.data_ptr(), workspace.numel()
    _run("rtl_attention", (*tensors, op, lp, shape, wp, size, flags), _here(q, k, v, q_starts, k_starts, k_lens), q, k=k, v=v,
         q_starts=q_starts, k_starts=k_starts, k_lens=k_lens)
    return (o, lse) if return_lse else o


def attention_backward(d_o, q, k, v, o, lse, causal: bool = False, scale: float = None, q_starts=None, k_starts=None,
                       k_lens=None, workspace=None):
    """Gradients (dq, dk, dv) of ``attention`` from d_o, its inputs, and the o and lse that it
    returned; arguments as there.  bf16 only.  Rows in no sequence, and behind the filled
    keys, are zeros."""
    torch = _torch()
    shape, tensors, n, k_starts = _shape(torch, q, k, v, scale, q_starts, k_starts, k_lens)
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"the backward pass is for bfloat16, got {q.dtype}")
    dp, op = _tensor(d_o, "d_o", q.dtype, q.dim()), _tensor(o, "o", q.dtype, q.dim())
    for name, t in (("d_o", d_o), ("o", o)):
        if t.shape != q.shape:
            raise ValueError(f"{name} must have q's shape {tuple(q.shape)}, got {tuple(t.shape)}")
    if lse.dtype is not torch.float32 or tuple(lse.shape) != _lse_shape(q) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {_lse_shape(q)}")
    dq, dk, dv = q.new_empty(q.shape), k.new_empty(k.shape), k.new_empty(k.shape)
    if n == 0:
        for t in (dq, dk, dv):
            t.zero_()
    workspace = _workspace(workspace, _fn("rtl_attention_backward_workspace_bytes")(shape), q.device)
    _run("rtl_attention_backward", (dp, *tensors, op, lse.data_ptr(), _new(dq), _new(dk), _new(dv), shape, workspace.data_ptr(),
                                    workspace.numel(), _CAUSAL if causal else 0),
         _here(q, k, v, d_o, o, lse, q_starts, k_starts, k_lens), q, k=k, v=v, d_o=d_o, o=o, lse=lse, q_starts=q_starts,
         k_starts=k_starts, k_lens=k_lens)
    return dq, dk, dv
