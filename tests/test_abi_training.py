"""The training entry points on the host, without a GPU: argument checks, and
the fp64 definitions that the GPU tests use against differences."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import training  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_plain as plain  # noqa: E402

OK, NULLP, SHAPE, MISAL, WS, NODEV, ARCH, HIP, FLAGS = range(9)
P = [0x10000 * i for i in range(1, 14)]
BIG = 1 << 40


def _no_gpu():
    return torch.cuda.device_count() == 0


def _pack(x=P[0], m=8, k=64, codes=P[1], exps=P[2], idx=P[3], stats=P[4]):
    return training._fn("rtl_checkpoint_pack")(x, m, k, codes, exps, idx, stats, None)


def _unpack(codes=P[1], exps=P[2], m=8, k=64, y=P[0]):
    return training._fn("rtl_checkpoint_unpack")(codes, exps, m, k, y, None)


def _back(g=P[0], codes=P[1], exps=P[2], idx=P[3], stats=P[4], w=P[5], a=P[6], b=P[7], m=8, n=64, k=128, r=16, dx=P[8],
          da=P[9], db=P[10], ws=P[11], size=BIG):
    return training._fn("rtl_sparse_linear_backward")(g, codes, exps, idx, stats, w, a, b, m, n, k, r, 1.0, dx, da, db, ws,
                                                      size, None)


def test_checkpoint_refusals():
    for call, ptrs in ((_pack, ("x", "codes", "exps", "idx", "stats")), (_unpack, ("codes", "exps", "y"))):
        for bad in (dict(m=-1), dict(k=0), dict(k=6), dict(k=-4), dict(m=1 << 31), dict(k=1 << 31), dict(m=1 << 20, k=1024)):
            assert call(**bad) == SHAPE, bad
        for p in ptrs:
            assert call(**{p: None}) == NULLP and call(**{p: 0x10008}) == MISAL
        assert call(m=0, **{p: None for p in ptrs}) == OK
        if _no_gpu():
            assert call() == NODEV


def test_backward_refusals():
    for bad in (dict(m=-1), dict(n=0), dict(n=6), dict(k=6), dict(k=0), dict(r=-1), dict(r=129), dict(m=1 << 23),
                dict(n=1 << 23), dict(r=0), dict(k=1 << 24)):
        assert _back(**bad) == SHAPE, bad
    for p in ("g", "codes", "exps", "idx", "stats", "w", "a", "b", "da", "db"):
        assert _back(**{p: None}) == NULLP, p
    for p in ("g", "codes", "exps", "idx", "stats", "w", "a", "b", "dx", "da", "db", "ws"):
        assert _back(**{p: 0x10004}) == MISAL, p
    need = training.backward_workspace_bytes(8, 64, 128, 16)
    assert _back(size=need - 1) == WS and _back(ws=None) == WS
    assert _back(dx=None, da=None, db=None, g=None) == OK
    assert _back(m=0, r=0, a=None, b=None, da=None, db=None, g=None, ws=None, size=0) == OK
    if _no_gpu():
        assert _back(size=need) == NODEV
        assert _back(dx=None, w=None) == NODEV
        assert _back(r=0, a=None, b=None, da=None, db=None) == NODEV
        assert _back(m=0, g=None, w=None, ws=None, size=0) == NODEV


def test_workspace_bytes():
    assert training.backward_workspace_bytes(0, 64, 128, 16) == 0
    for bad in ((-1, 64, 128, 16), (8, 62, 128, 16), (8, 64, 126, 16), (8, 64, 128, 129), (8, 64, 128, -1), (1 << 23, 64, 128, 0)):
        assert training.backward_workspace_bytes(*bad) == 0
    for m, n, k, r in ((1, 4, 4, 0), (8, 64, 128, 16), (4096, 12288, 3072, 64)):
        assert training.backward_workspace_bytes(m, n, k, r) >= 4 * m * k + 8 * m * r


def test_definitions_agree_with_differences():
    m, n, k, r, alpha = 6, 10, 16, 3, 0.7
    rng = np.random.default_rng(1)
    x, w, a, b, g = (rng.standard_normal(s) for s in ((m, k), (n, k), (r, k), (n, r), (m, n)))
    x[2] = 0                                             # s is 1 there and has no derivative: left out below
    order = np.argsort(-np.abs(x).reshape(m, -1, 4), axis=-1, kind="stable")
    mk = np.zeros((m, k // 4, 4))
    np.put_along_axis(mk, order[..., :2], 1.0, -1)
    mk = mk.reshape(m, k)
    lk = (mk * np.abs(x)).sum(1)
    s = np.where(lk > 0, np.abs(x).sum(1) / np.where(lk > 0, lk, 1), 1.0)
    (dx, da, db), _ = plain.backward(g, x, mk, s, lk, w.T, a, b, alpha)
    loss = lambda *p: (g * plain.forward(p[0], mk, w, p[1], p[2], alpha)).sum()  # noqa: E731
    for which, (point, grad) in enumerate(((x, dx), (a, da), (b, db))):
        for _ in range(5):
            step = rng.standard_normal(point.shape)
            if which == 0:
                step[2] = 0
            lo, hi = [x, a, b], [x, a, b]
            lo[which], hi[which] = point - 1e-6 * step, point + 1e-6 * step
            diff = (loss(*hi) - loss(*lo)) / 2e-6
            assert abs(diff - (grad * step).sum()) <= 1e-6 * max(1.0, np.abs(grad * step).sum())


def test_pack_definition():
    x = np.array([[1.0, -1.0, 0.5, 0.0] + [2.0 ** -9] * 4])
    codes, exps = plain.pack(x)
    assert exps[0, 0] == 127 and codes[0].tolist() == [64, -64, 32, 0, 0, 0, 0, 0]
    x = np.array([[2.0 - 2.0 ** -7, 1.0, 0, 0]])         # 127.5 steps: clamped
    codes, exps = plain.pack(x)
    assert codes[0].tolist() == [127, 64, 0, 0] and (np.abs(plain.values(codes, exps) - x) <= 2.0 ** -7).all()
    assert plain.mask(np.array([[0x4e]], np.uint8), 8)[0].tolist() == [0, 0, 1, 1, 1, 1, 0, 0]


def test_binding_refusals():
    with pytest.raises(ValueError):
        training.checkpoint(torch.zeros(2, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        training.unpack(torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.uint8))
