"""Linear layers of few rows with 4-bit weights and group scales
(include/rtlynx_w4.h): ``pack`` lays a weight out once, ``linear`` multiplies.
Argument marshalling only, as in the package's other bindings.
"""
from __future__ import annotations

import ctypes

from . import _as_2d, _check, _here, _no_graph, _on, _out, _separate, _stream, _torch, lib

__all__ = ["Weight", "pack", "linear", "packed_bytes", "GROUPS", "MAX_ROWS"]

GROUPS = (32, 64, 128)
MAX_ROWS = 1 << 20
_ZEROS = 0x1

_c_i64, _c_vp, _c_size, _c_u32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32
_SIGNATURES = {
    "rtl_w4_packed_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_u32]),
    "rtl_w4_pack": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_u32, _c_vp, _c_size, _c_vp]),
    "rtl_w4_linear": (ctypes.c_int, [_c_vp, _c_vp, _c_size, _c_i64, _c_i64, _c_i64, _c_i64, _c_u32, _c_vp, _c_vp]),
}


def _fn(name):
    fn = getattr(lib(), name)
    if fn.argtypes is None:
        fn.restype, fn.argtypes = _SIGNATURES[name]
    return fn


def packed_bytes(n: int, k: int, group: int, zeros: bool = False) -> int:
    return int(_fn("rtl_w4_packed_bytes")(n, k, group, _ZEROS if zeros else 0))


class Weight:
    """A weight [n, k] laid out by ``pack``: contiguous uint8 bytes on the device
    (one read back from a file is put together here; its size is checked by the
    library)."""

    def __init__(self, packed, n: int, k: int, group: int, zeros: bool):
        if packed.dtype != _torch().uint8:
            raise TypeError(f"packed must be uint8, got {packed.dtype}")
        if not packed.is_cuda or not packed.is_contiguous():
            raise ValueError("packed must be a contiguous device tensor")
        self.packed, self.n, self.k, self.group, self.zeros = packed, n, k, group, zeros


def pack(codes, scales, zeros=None, group: int = 128) -> Weight:
    """Lays out codes [n, k / 2] uint8 (channel 2i in the low half of byte i),
    scales [n, k / group] bf16 and, optionally, zero points [n, k / group]
    uint8 (0..15; 8 throughout without them) for ``linear``."""
    torch = _torch()
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group}")
    if codes.dtype != torch.uint8 or codes.dim() != 2:
        raise TypeError("codes must be uint8 [n, k / 2]")
    n, k = codes.shape[0], 2 * codes.shape[1]
    if n < 1 or k < 1 or k % group:
        raise ValueError(f"a weight [{n}, {k}] has no whole groups of {group} channels")
    for name, t, dt in (("codes", codes, torch.uint8), ("scales", scales, torch.bfloat16), ("zeros", zeros, torch.uint8)):
        if t is None:
            continue
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous device tensor")
        if name != "codes" and tuple(t.shape) != (n, k // group):
            raise ValueError(f"{name} must have shape {(n, k // group)}, got {tuple(t.shape)}")
    flags = _ZEROS if zeros is not None else 0
    packed = torch.empty((packed_bytes(n, k, group, zeros is not None),), dtype=torch.uint8, device=codes.device)
    with _on(codes.device, scales=scales, zeros=zeros):
        st = _fn("rtl_w4_pack")(codes.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                                n, k, group, flags, packed.data_ptr(), packed.numel(), _stream())
    _check(st, "rtl_w4_pack")
    return Weight(packed, n, k, group, zeros is not None)


def linear(x, weight: Weight, out=None):
    """y [..., n] bf16 = x [..., k] bf16 times the weight: made for 1 to 64
    rows, accepts up to ``MAX_ROWS``.  x must be finite; ``out`` shares no memory
    with it.  For inference: the result has no autograd graph."""
    if x.requires_grad:
        _no_graph("w4.linear", "it has none", x)
    x2 = _as_2d(x, "x")
    m, k = x2.shape
    if k != weight.k:
        raise ValueError(f"the weight has {weight.k} input channels, x has {k}")
    y = x2.new_empty((*x.shape[:-1], weight.n)) if out is None else _out(out, m, weight.n, x.shape[:-1], x2.device)
    packed = weight.packed
    if out is not None:
        _separate(out, x=x2, weight=packed)
    args = (x2.data_ptr(), packed.data_ptr(), packed.numel(), m, weight.n, k, weight.group,
            _ZEROS if weight.zeros else 0, y.data_ptr())
    stream = _here(x2, packed)
    if stream is None:
        with _on(x2.device, weight=packed):
            st = _fn("rtl_w4_linear")(*args, _stream())
    else:
        st = _fn("rtl_w4_linear")(*args, stream)
    _check(st, "rtl_w4_linear")
    return y if out is None else y.view(*x.shape[:-1], weight.n)
