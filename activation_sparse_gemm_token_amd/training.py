"""Training the LoRA branch of the sparse layer (include/rtlynx_train.h): the
layer's input kept in 8 bits, and the backward pass that reads it.

    y    = sparse_linear(x, w, a, b, alpha)         # forward
    kept = training.checkpoint(x, fine=True)        # instead of keeping x
    dx, da, db = training.sparse_linear_backward(dy, kept, w_t, a, b, alpha)

No call records an autograd graph: a model calls these in the forward and backward
of its own ``torch.autograd.Function``.  The gradients are those of ``sparse_linear``
(the default layer); dense layers and the compensation and LoRA-input variants of
``layers.LayerPolicy`` have none here.  Argument marshalling only, as in the
package's other bindings.
"""
from __future__ import annotations

import ctypes

from . import _as_2d, _check, _here, _on, _out, _separate, _stream, _torch, _workspace, lib

__all__ = ["Checkpoint", "checkpoint", "unpack", "sparse_linear_backward", "backward_workspace_bytes",
           "backward_form"]

_c_i64, _c_vp, _c_size, _c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_SIGNATURES = {
    "rtl_checkpoint_pack": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "rtl_checkpoint_pack_fine": (_c_int, [_c_vp, _c_i64, _c_i64] + [_c_vp] * 6),
    "rtl_checkpoint_unpack": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "rtl_checkpoint_unpack_fine": (_c_int, [_c_vp] * 4 + [_c_i64, _c_i64, _c_vp, _c_vp]),
    "rtl_sparse_linear_backward_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "rtl_sparse_linear_backward_form": (_c_int, [_c_i64] * 4 + [ctypes.POINTER(_c_i64)]),
    "rtl_sparse_linear_backward": (_c_int, [_c_vp] * 8 + [_c_i64] * 4 + [ctypes.c_float] + [_c_vp] * 4 +
                                   [_c_size, _c_vp]),
    "rtl_sparse_linear_backward_fine": (_c_int, [_c_vp] * 9 + [_c_i64] * 4 + [ctypes.c_float] + [_c_vp] * 4 +
                                        [_c_size, _c_vp]),
}


def _fn(name):
    fn = getattr(lib(), name)
    if fn.argtypes is None:
        fn.restype, fn.argtypes = _SIGNATURES[name]
    return fn


def _run(name, args, t, **tensors):
    """Entry point ``name`` on t's device, which the named tensors share, and
    its current stream."""
    stream = _here(t, *tensors.values())
    if stream is None:
        with _on(t.device, **tensors):
            st = _fn(name)(*args, _stream())
    else:
        st = _fn(name)(*args, stream)
    _check(st, name)


class Checkpoint:
    """A layer's input [m, k] in 8 bits: ``codes`` int8 [m, k] times
    2^(``exps`` - 133) per 32 channels (uint8 [m, ceil(k / 32)]), the kept
    channels ``idx`` uint8 [m, ceil(k / 8)] and ``stats`` fp32 [m, 2] (the
    token's scale, the L1 norm of its kept channels).  ``lead`` is the shape of
    x without its channels.  With ``pruned_exps``, shaped like ``exps``, the pruned
    channels' codes count steps of 2^(``pruned_exps`` - 133)."""

    def __init__(self, codes, exps, idx, stats, lead=None, pruned_exps=None):
        torch = _torch()
        if codes.dim() != 2:
            raise ValueError("codes must be [m, k]")
        m, k = codes.shape
        if k < 4 or k % 4:
            raise ValueError(f"k must be a multiple of 4, got {k}")
        for name, t, dtype, shape in (("codes", codes, torch.int8, (m, k)),
                                      ("exps", exps, torch.uint8, (m, (k + 31) // 32)),
                                      ("idx", idx, torch.uint8, (m, (k + 7) // 8)),
                                      ("stats", stats, torch.float32, (m, 2)),
                                      ("pruned_exps", pruned_exps, torch.uint8, (m, (k + 31) // 32))):
            if t is None and name == "pruned_exps":
                continue
            if t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous device tensor")
            if t.device != codes.device:
                raise ValueError(f"{name} is on {t.device}, codes on {codes.device}")
        self._set(codes, exps, idx, stats, (m,) if lead is None else tuple(lead), pruned_exps)

    def _set(self, codes, exps, idx, stats, lead, pruned_exps):
        self.codes, self.exps, self.idx, self.stats, self.lead = codes, exps, idx, stats, lead
        self.pruned_exps = pruned_exps
        self.m, self.k = codes.shape

    @classmethod
    def _made(cls, codes, exps, idx, stats, lead, pruned_exps):
        """A checkpoint of tensors that ``checkpoint`` made: nothing to check."""
        kept = cls.__new__(cls)
        kept._set(codes, exps, idx, stats, tuple(lead), pruned_exps)
        return kept

    def unpack(self, out=None):
        """The stored values [*lead, k] in bf16 (exact)."""
        codes = self.codes
        if out is not None:
            y = _out(out, self.m, self.k, self.lead, codes.device).view(*self.lead, self.k)
            _separate(y, codes=codes, exps=self.exps, idx=self.idx)
            if self.pruned_exps is not None:
                _separate(y, pruned_exps=self.pruned_exps)
        else:
            y = codes.new_empty((*self.lead, self.k), dtype=_torch().bfloat16)
        if self.pruned_exps is None:
            _run("rtl_checkpoint_unpack", (codes.data_ptr(), self.exps.data_ptr(), self.m, self.k, y.data_ptr()), codes)
        else:
            _run("rtl_checkpoint_unpack_fine", (codes.data_ptr(), self.exps.data_ptr(), self.pruned_exps.data_ptr(),
                                                self.idx.data_ptr(), self.m, self.k, y.data_ptr()), codes)
        return y


def checkpoint(x, fine: bool = False) -> Checkpoint:
    """Keeps x [..., k] (bf16, finite) in 8 bits for the backward pass.

    ``fine`` keeps a second exponent per 32 channels, of the pruned ones, and their
    signs (1.19 bytes a channel instead of 1.16).  Where a few channels are far
    larger than the rest, the one exponent makes more than half of the pruned
    channels zero, and with 8 % of them large dA and dB are off by 17 % and dX by 9 %;
    ``fine`` makes it 1.9 % and 0.2 %.  With activations of one scale both are within
    3 % (include/rtlynx_train.h)."""
    torch = _torch()
    x2 = _as_2d(x, "x")
    m, k = x2.shape
    codes = torch.empty_like(x2, dtype=torch.int8)
    exps = x2.new_empty((m, (k + 31) // 32), dtype=torch.uint8)
    idx = x2.new_empty((m, (k + 7) // 8), dtype=torch.uint8)
    stats = x2.new_empty((m, 2), dtype=torch.float32)
    pruned_exps = torch.empty_like(exps) if fine else None
    if fine:
        _run("rtl_checkpoint_pack_fine", (x2.data_ptr(), m, k, codes.data_ptr(), exps.data_ptr(), pruned_exps.data_ptr(),
                                          idx.data_ptr(), stats.data_ptr()), x2)
    else:
        _run("rtl_checkpoint_pack", (x2.data_ptr(), m, k, codes.data_ptr(), exps.data_ptr(), idx.data_ptr(),
                                     stats.data_ptr()), x2)
    return Checkpoint._made(codes, exps, idx, stats, x.shape[:-1], pruned_exps)


def unpack(codes, exps, out=None):
    """bf16 values [m, k] of int8 codes [m, k] and exponents [m, ceil(k / 32)] (one
    exponent per block; ``Checkpoint.unpack`` serves both forms)."""
    torch = _torch()
    if codes.dtype != torch.int8 or exps.dtype != torch.uint8:
        raise TypeError("codes must be int8 and exps uint8")
    if codes.dim() != 2 or tuple(exps.shape) != (codes.shape[0], (codes.shape[1] + 31) // 32):
        raise ValueError("codes must be [m, k] and exps [m, ceil(k / 32)]")
    if not codes.is_cuda or not codes.is_contiguous() or not exps.is_contiguous():
        raise ValueError("codes and exps must be contiguous device tensors")
    m, k = codes.shape
    y = _out(out, m, k, (m,), codes.device)
    if out is not None:
        _separate(out, codes=codes, exps=exps)
    _run("rtl_checkpoint_unpack", (codes.data_ptr(), exps.data_ptr(), m, k, y.data_ptr()), codes, exps=exps)
    return y


def backward_workspace_bytes(m: int, n: int, k: int, r: int) -> int:
    return int(_fn("rtl_sparse_linear_backward_workspace_bytes")(m, n, k, r))


def backward_form(m: int, n: int, k: int, r: int):
    """Which kernels ``sparse_linear_backward`` takes at these sizes: (tile columns
    of G W, its ranges, its row length, channels per range over n and over k,
    tokens per range)."""
    form = (_c_i64 * 6)()
    _check(_fn("rtl_sparse_linear_backward_form")(m, n, k, r, form), "rtl_sparse_linear_backward_form")
    return tuple(form)


def sparse_linear_backward(g, kept: Checkpoint, w_t, lora_a=None, lora_b=None, lora_scale: float = 1.0,
                           need_dx: bool = True, need_lora: bool = True, workspace=None):
    """Gradients of ``sparse_linear`` from g = dL/dy [..., n] and the input's
    checkpoint: (dx [..., k], da [r, k], db [n, r]), bf16, None where not
    asked for (da and db are None without a LoRA branch).

    ``w_t`` [k, n] is the frozen weight transposed, laid out once
    (``w.t().contiguous()``); it may be None when ``need_dx`` is False."""
    g2 = _as_2d(g, "g")
    m, n = g2.shape
    k = kept.k
    if m != kept.m:
        raise ValueError(f"g has {m} tokens, the checkpoint {kept.m}")
    if w_t is None and need_dx:
        raise ValueError("dx needs w_t")
    if w_t is not None:
        w_t = _as_2d(w_t, "w_t")
        if tuple(w_t.shape) != (k, n):
            raise ValueError(f"w_t must be [{k}, {n}], got {tuple(w_t.shape)}")
    r = 0
    if lora_a is not None or lora_b is not None:
        if lora_a is None or lora_b is None:
            raise ValueError("lora_a and lora_b go together")
        lora_a, lora_b = _as_2d(lora_a, "lora_a"), _as_2d(lora_b, "lora_b")
        r = lora_a.shape[0]
        if lora_a.shape[1] != k or tuple(lora_b.shape) != (n, r):
            raise ValueError(f"LoRA shapes {tuple(lora_a.shape)}, {tuple(lora_b.shape)} do not match K={k}, N={n}")
    dev = g2.device
    lead = g.shape[:-1]
    dx = g2.new_empty((*lead, k)) if need_dx else None
    lora = need_lora and r > 0
    da = g2.new_empty((r, k)) if lora else None
    db = g2.new_empty((n, r)) if lora else None
    workspace = _workspace(workspace, backward_workspace_bytes(m, n, k, r), dev)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    fine = () if kept.pruned_exps is None else (kept.pruned_exps.data_ptr(),)
    _run("rtl_sparse_linear_backward_fine" if fine else "rtl_sparse_linear_backward",
         (g2.data_ptr(), kept.codes.data_ptr(), kept.exps.data_ptr(), *fine, kept.idx.data_ptr(), kept.stats.data_ptr(),
          ptr(w_t), ptr(lora_a) if r else None, ptr(lora_b) if r else None, m, n, k, r, float(lora_scale), ptr(dx),
          ptr(da), ptr(db), workspace.data_ptr(), workspace.numel()),
         g2, kept=kept.codes, w_t=w_t, lora_a=lora_a, lora_b=lora_b)
    return dx, da, db
