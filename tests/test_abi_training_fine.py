"""The checkpoint with a step of its own for the pruned channels, on the host: argument
checks, and what either form loses of the gradients, by their definitions in fp64."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import training  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_plain as plain  # noqa: E402
from fine_plain import pack_fine, select, values_fine  # noqa: E402

OK, NULLP, SHAPE, MISAL, WS, NODEV = range(6)
P = [0x10000 * i for i in range(1, 15)]


def _no_gpu():
    return torch.cuda.device_count() == 0


def _pack(x=P[0], m=8, k=64, codes=P[1], exps=P[2], pruned=P[3], idx=P[4], stats=P[5]):
    return training._fn("rtl_checkpoint_pack_fine")(x, m, k, codes, exps, pruned, idx, stats, None)


def _unpack(codes=P[1], exps=P[2], pruned=P[3], idx=P[4], m=8, k=64, y=P[0]):
    return training._fn("rtl_checkpoint_unpack_fine")(codes, exps, pruned, idx, m, k, y, None)


def _back(g=P[0], codes=P[1], exps=P[2], pruned=P[12], idx=P[3], stats=P[4], w=P[5], a=P[6], b=P[7], m=8, n=64, k=128,
          r=16, dx=P[8], da=P[9], db=P[10], ws=P[11], size=1 << 40):
    return training._fn("rtl_sparse_linear_backward_fine")(g, codes, exps, pruned, idx, stats, w, a, b, m, n, k, r, 1.0, dx,
                                                           da, db, ws, size, None)


@pytest.mark.parametrize("call,ptrs", [(_pack, ("x", "codes", "exps", "pruned", "idx", "stats")),
                                       (_unpack, ("codes", "exps", "pruned", "idx", "y")),
                                       (_back, ("g", "codes", "exps", "pruned", "idx", "stats", "w", "a", "b"))])
def test_refusals(call, ptrs):
    for bad in (dict(m=-1), dict(k=0), dict(k=6), dict(m=1 << 31), dict(k=1 << 31)):
        assert call(**bad) == SHAPE, bad
    for p in ptrs:
        assert call(**{p: None}) == NULLP and call(**{p: 0x10008}) == MISAL, p
    if call is not _back:
        assert call(m=0, **{p: None for p in ptrs}) == OK
    if _no_gpu():
        assert call() == NODEV


def test_definition():
    x = np.array([[4.0, -2.0, 2.0 ** -9, -2.0 ** -12, 8.0, 1.0, 0.0, 3 * 2.0 ** -17]])
    codes, exps, pruned = pack_fine(x, select(x))
    assert exps[0, 0] == 130 and pruned[0, 0] == 118               # 8 and 2^-9
    assert codes[0].tolist() == [32, -16, 64, -8, 64, 8, 0, 1]     # 0.75 steps is 1; so is any smaller one
    assert np.array_equal(values_fine(codes, exps, pruned, select(x))[0, :6], x[0, :6])
    x[0, 7] = -2.0 ** -30
    assert pack_fine(x, select(x))[0][0, 7] == -1


@pytest.mark.parametrize("law,fine,da,dx", [("mixture", False, 0.17, 0.09), ("mixture", True, 0.019, 0.003),
                                            ("gauss", False, 0.013, 0.006), ("gauss", True, 0.008, 0.001)])
def test_what_the_gradients_lose(law, fine, da, dx):
    """The figures that the header states: relative error of the gradients formed from
    the stored values against those of x itself, in the 2-norm."""
    m, n, k, r = 256, 256, 1024, 16
    rng = np.random.default_rng(3)
    bf = lambda a: torch.from_numpy(a).bfloat16().double().numpy()  # noqa: E731
    z = rng.standard_normal((m, k))
    x = bf(z if law == "gauss" else np.where(rng.random((m, k)) < 0.08, 4 * z, 0.05 * z))
    g, w_t, a, b = (bf(std * rng.standard_normal(s)) for std, s in ((.01, (m, n)), (.02, (k, n)), (.01, (r, k)), (.01, (n, r))))
    mk = select(x)
    lk = (mk * np.abs(x)).sum(1)
    s = np.abs(x).sum(1) / lk
    stored = values_fine(*pack_fine(x, mk), mk) if fine else plain.values(*plain.pack(x))
    want, _ = plain.backward(g, x, mk, s, lk, w_t, a, b, 1.0)
    got, _ = plain.backward(g, stored, mk, s, lk, w_t, a, b, 1.0)
    off = [np.linalg.norm(p - q) / np.linalg.norm(q) for p, q in zip(got, want)]
    for have, stated in zip(off, (dx, da, da)):                    # another draw of the law: a third either way
        assert have <= stated * 4 / 3
    if law == "mixture" and not fine:
        assert min(off[0] / dx, off[1] / da, off[2] / da) >= 2 / 3
