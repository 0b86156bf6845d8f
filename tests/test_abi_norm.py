"""rtl_layer_norm and its binding on the host, without a GPU: argument checks."""
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import norm  # noqa: E402

OK, NULLP, SHAPE, MISAL, WS, NODEV, ARCH, HIP, FLAGS = range(9)
P, P2, P3, P4, P5, P6, P7, P8 = (0x10000 * i for i in range(1, 9))


def _forward(x=P, b=2, t=3, c=64, xb=192, xt=64, w=P2, wb=0, bias=P3, bb=0, y=P4, yb=192, yt=64, mean=P5, rstd=P6, flags=0):
    return norm._fn("rtl_layer_norm")(x, b, t, c, xb, xt, w, wb, bias, bb, 0.0, 1e-5, y, yb, yt, mean, rstd, flags, None)


def _backward(dy=P, x=P2, mean=P3, rstd=P4, b=2, t=3, c=64, s=64, w=P5, wb=0, groups=1, dx=P6, dw=P7, db=P8, ws=P, wsb=1 << 24,
              flags=0):
    return norm._fn("rtl_layer_norm_backward")(dy, 192, s, x, 192, s, mean, rstd, b, t, c, w, wb, 0.0, groups, dx, 192, s, dw,
                                               db, ws, wsb, flags, None)


def _no_gpu():
    return torch.cuda.device_count() == 0


def test_forward_refusals():
    for bad in (3, 0x20, 0x100):
        assert _forward(flags=bad) == FLAGS
    for bad in (dict(b=-1), dict(t=-1), dict(c=0), dict(c=32769), dict(xb=-1), dict(xt=1 << 40), dict(yt=-64), dict(wb=-1),
                dict(bb=1 << 40), dict(b=1 << 30, t=4), dict(t=1 << 31)):
        assert _forward(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(y=None), dict(w=None), dict(mean=None), dict(rstd=None)):
        assert _forward(**bad) == NULLP, bad
    for bad in (dict(x=P + 1), dict(y=P4 + 1), dict(w=P2 + 1), dict(bias=P3 + 1), dict(mean=P5 + 2), dict(x=P + 2, flags=2),
                dict(w=P2 + 2, flags=0x10)):
        assert _forward(**bad) == MISAL, bad
    assert _forward(b=0, x=None, y=None) == OK and _forward(t=0) == OK
    if _no_gpu():
        assert _forward() == NODEV and _forward(w=None, bias=None, mean=None, rstd=None, flags=0x12) == NODEV


def test_backward_refusals():
    for bad in (3, 0x20, 0x100):
        assert _backward(flags=bad) == FLAGS
    for bad in (dict(b=-1), dict(c=0), dict(c=32769), dict(s=-1), dict(groups=3), dict(groups=-1), dict(wb=-1), dict(t=1 << 31)):
        assert _backward(**bad) == SHAPE, bad
    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dw=None), dict(db=None)):
        assert _backward(**bad) == NULLP, bad
    for bad in (dict(dy=P + 1), dict(x=P2 + 1), dict(dx=P6 + 1), dict(dw=P7 + 1), dict(mean=P3 + 1), dict(ws=P + 8),
                dict(dw=P7 + 2, flags=0x10)):
        assert _backward(**bad) == MISAL, bad
    need = norm.backward_workspace_bytes(2, 300, 64, 1)
    assert need > 0 and _backward(t=300, wsb=need - 1) == WS and _backward(t=300, ws=None) == WS
    assert norm.backward_workspace_bytes(2, 300, 64, 2) > 0 and norm.backward_workspace_bytes(2, 300, 64, 3) == 0
    assert norm.backward_workspace_bytes(2, 3, 64, 1) == 0                  # one workgroup has all rows
    assert _backward(b=0, groups=0) == OK and _backward(t=0, dw=None, db=None, dy=None) == OK
    assert _backward(dx=None, dw=None, db=None) == OK
    if _no_gpu():
        assert _backward() == NODEV and _backward(dw=None, db=None, ws=None) == NODEV and _backward(t=0) == NODEV


def test_binding_needs_device_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        norm.layer_norm(x)
    with pytest.raises(TypeError):
        norm.layer_norm(x.double())
