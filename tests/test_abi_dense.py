"""rtl_linear and its binding on the host, without a GPU: argument checks."""
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import dense  # noqa: E402

OK, NULLP, SHAPE, MISAL, WS, NODEV, ARCH, HIP, FLAGS = range(9)
P = [0x10000 * i for i in range(1, 12)]


def _forward(x=P[0], w=P[1], bias=P[2], gate=P[3], rows=1, stride=0, res=P[4], m=64, n=128, k=64, y=P[5], z=P[6], ws=P[7],
             wsb=1 << 30, flags=0):
    return dense._fn("rtl_linear")(x, w, bias, gate, rows, stride, res, m, n, k, y, z, ws, wsb, flags, None)


def _backward(dy=P[0], x=P[1], w=P[2], z=P[3], gate=P[4], rows=1, stride=0, m=64, n=128, k=64, dx=P[5], dw=P[6], db=P[7],
              dg=P[8], ws=P[9], wsb=1 << 30, flags=0x10):
    return dense._fn("rtl_linear_backward")(dy, x, w, z, gate, rows, stride, m, n, k, dx, dw, db, dg, ws, wsb, flags, None)


def _no_gpu():
    return torch.cuda.device_count() == 0


@pytest.mark.parametrize("call", [_forward, _backward])
def test_refusals(call):
    for bad in (0x2, 0x3, 0x40, 0x80, 0x102):
        assert call(flags=bad) == FLAGS, bad
    for bad in (dict(m=-1), dict(n=-1), dict(k=0), dict(k=4), dict(k=60), dict(m=1 << 25), dict(n=1 << 25), dict(m=1 << 20, n=1 << 10),
                dict(rows=0), dict(rows=3), dict(rows=-1), dict(stride=-1), dict(stride=1 << 40), dict(rows=1 << 17, m=1 << 17)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=P[0] + 8), dict(w=P[1] + 8), dict(z=P[6] + 8), dict(gate=P[3] + 1), dict(ws=P[7] + 8)):
        assert call(**bad) == MISAL, bad
    for bad in (dict(x=None), dict(w=None)):
        assert call(**bad) == NULLP, bad


def test_forward():
    assert _forward(y=None) == NULLP and _forward(y=P[5] + 8) == MISAL and _forward(res=P[4] + 8) == MISAL
    assert _forward(bias=P[2] + 1) == MISAL
    need = dense.workspace_bytes(64, 128, 4096)
    assert need > 0 and _forward(k=4096, wsb=need - 1) == WS and _forward(k=4096, ws=None) == WS
    assert dense.workspace_bytes(64, 128, 60) == 0 and dense.workspace_bytes(8, 128, 4096) == 0
    assert _forward(m=0, x=None) == OK and _forward(n=0) == OK
    assert _forward(gate=None, rows=7, m=0) == OK                  # no gate: its rows do not count
    if _no_gpu():
        assert _forward() == NODEV and _forward(bias=None, gate=None, res=None, z=None, flags=0x31) == NODEV
        assert _forward(m=8, k=4096, ws=None, wsb=0) == NODEV


def test_backward():
    assert _backward(dy=None) == NULLP and _backward(z=None) == NULLP and _backward(z=None, flags=0) == NULLP
    assert _backward(x=None, dw=None, w=None, dx=None, wsb=0) == WS
    need = dense.backward_workspace_bytes(64, 128, 64)
    assert need >= 2 * 64 * 128 and _backward(wsb=need - 1) == WS and _backward(ws=None) == WS
    assert dense.backward_workspace_bytes(64, 128, 64, 3) == 0
    for bad in (dict(dx=P[5] + 8), dict(dw=P[6] + 8), dict(db=P[7] + 1), dict(dg=P[8] + 1), dict(dy=P[0] + 2)):
        assert _backward(**bad) == MISAL, bad
    assert _backward(dx=None, dw=None, db=None, dg=None) == OK and _backward(n=0, m=0) == OK
    if _no_gpu():
        assert _backward() == NODEV and _backward(z=None, dg=None, flags=1) == NODEV and _backward(m=0, dy=None, z=None) == NODEV


def test_binding_needs_device_tensors():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dense.linear(x, w)
    with pytest.raises(TypeError):
        dense.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        dense.linear(x, w, activation="relu6")


def test_widths():
    for bad in (dict(m=1, n=1 << 25, k=8), dict(m=1, n=8, k=1 << 25)):
        assert _forward(**bad) == SHAPE and _backward(**bad) == SHAPE and dense.workspace_bytes(bad["m"], bad["n"], bad["k"]) == 0, bad
    if _no_gpu():
        assert _forward(m=1, n=(1 << 25) - 8, k=8) == NODEV
