"""rtl_rope and its binding on the host, without a GPU: argument checks and
the frequency tables."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import rotary  # noqa: E402

OK, NULLP, SHAPE, MISAL, WS, NODEV, ARCH, HIP, FLAGS = range(9)
P, P2, P3, P4 = 0x10000, 0x20000, 0x30000, 0x40000


def _call(tensors=None, count=1, b=2, t=3, d=64, rot=64, pos=P3, pb=3, pt=1, axes=1, pairs=None, freq=P4, flags=0,
          **kw):
    one = rotary._Tensor(kw.get("x", P), kw.get("y", P2), kw.get("heads", 4), 768, 256, 64, 768, 256, 64)
    if "stride" in kw:
        one.x_token_stride = kw["stride"]
    arr = (rotary._Tensor * 2)(one, one) if tensors is None else tensors
    ap = (ctypes.c_int32 * len(pairs))(*pairs) if pairs is not None else None
    return rotary._fn()(arr, count, b, t, d, rot, pos, pb, pt, axes, ap, freq, 1.0, flags, None)


def _no_gpu():
    return torch.cuda.device_count() == 0


def test_refusals():
    for bad in (dict(flags=3), dict(flags=0x40), dict(flags=0x100)):
        assert _call(**bad) == FLAGS, bad
    for bad in (dict(count=0), dict(count=3), dict(b=-1), dict(t=-1), dict(d=0), dict(d=1025), dict(rot=63),
                dict(rot=66), dict(rot=-2), dict(axes=0), dict(axes=5, pairs=[32, 0, 0, 0, 0]),
                dict(axes=2, pairs=[16, 15]), dict(axes=2, pairs=[33, -1]), dict(axes=2, pairs=[40, 0]),
                dict(axes=1, pairs=[31]), dict(heads=-1), dict(stride=1 << 40), dict(pb=1 << 40), dict(b=1 << 30, t=4)):
        assert _call(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(y=None), dict(pos=None), dict(freq=None), dict(axes=2)):
        assert _call(**bad) == NULLP, bad
    assert rotary._fn()(None, 1, 1, 1, 64, 64, P, 1, 1, 1, None, P, 1.0, 0, None) == NULLP
    for bad in (dict(x=P + 1), dict(y=P2 + 1), dict(x=P + 2, flags=2), dict(pos=P3 + 4), dict(freq=P4 + 4)):
        assert _call(**bad) == MISAL, bad


def test_empty_calls_and_valid_ones():
    assert _call(b=0) == OK and _call(t=0) == OK and _call(heads=0) == OK
    if _no_gpu():
        assert _call() == NODEV
        assert _call(x=P + 2) == NODEV
        assert _call(rot=0, pos=None, freq=None) == NODEV
        assert _call(count=2, axes=3, pairs=[0, 16, 16], flags=0x32) == NODEV


def test_frequency_tables():
    f = rotary.frequencies(8, base=10000.0)
    assert f.dtype == torch.float64 and f[0] == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14, atol=0)
    assert torch.allclose(rotary.frequencies(8, linear=4.0), f / 4, rtol=1e-15, atol=0)
    n = rotary.frequencies(8, ntk=4.0)
    assert n[0] == 1.0 and abs(n[-1] / f[-1] - 0.25) < 1e-12
    g, scale = rotary.frequencies_by_parts(128, 8.0, 4096)
    full = rotary.frequencies(128)
    turns = 4096 * full / (2 * math.pi)
    assert scale == 0.1 * math.log(8.0) + 1.0
    assert torch.equal(g[turns > 40], full[turns > 40])
    assert torch.allclose(g[turns < 0.8], full[turns < 0.8] / 8, rtol=1e-14, atol=0)
    assert ((g <= full) & (g >= full / 8 * (1 - 1e-14))).all()
    for bad in (lambda: rotary.frequencies(7), lambda: rotary.frequencies(8, base=0.0),
                lambda: rotary.frequencies_by_parts(8, 0.5, 10)):
        with pytest.raises(ValueError):
            bad()
    assert rotary.frequencies(0).shape == (0,) and rotary.frequencies(2, ntk=2.0)[0] == 1.0


def test_binding_needs_device_tensors_and_known_layouts():
    x, pos, f = torch.zeros(2, 3, 8), torch.zeros(2, dtype=torch.int64), rotary.frequencies(8)
    with pytest.raises(ValueError):
        rotary.rope(x, pos, f)
    with pytest.raises(ValueError):
        rotary.rope(x, pos, f, layout="other")
    with pytest.raises(TypeError):
        rotary.rope(x.double(), pos, f)
    with pytest.raises(ValueError):
        rotary.rope(x[0], pos, f)


def test_overlap_rules():
    base = torch.zeros(2, 5, 9, 16)
    q, k, v = base[:, :, :4], base[:, :, 4:6], base[:, :, 6:]
    assert rotary._apart(q, k) and rotary._apart(k, q) and rotary._apart(k, v)
    assert not rotary._apart(q, base[:, :, 3:5]) and not rotary._apart(q, q)
    assert not rotary._apart(q, base[:, :, :4].transpose(1, 2))
    assert rotary._apart(base[:1], base[1:])
    assert rotary._same(q, base[:, :, :4]) and not rotary._same(q, k)
    assert rotary._distinct(q) and rotary._distinct(q.transpose(1, 2))
    assert not rotary._distinct(torch.zeros(2, 1, 4).expand(2, 3, 4))
    assert not rotary._distinct(torch.zeros(20).as_strided((3, 4), (2, 1)))
