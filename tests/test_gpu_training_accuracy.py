"""How exact the training calls are: what is carried between the products, the
checkpoint's own error in the gradients, and its statistics."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import training  # noqa: E402
from workloads import gen  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_plain as plain  # noqa: E402

DEV = "cuda:0"


def to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).bfloat16().to(DEV)


@pytest.mark.parametrize("m,r", [(1, 2), (1, 40), (70, 3), (2, 100), (600, 33), (40, 128)])
def test_u_and_t_keep_fp32s_bits(m, r):
    """One token whose U and T are 1 + 2^-8 +- 2^-20 times powers of two, exact in
    fp32 in any order: the last bit decides to which side the result rounds, so
    whatever held them in fewer than 21 bits between the products would miss it."""
    n, k, at = 12, 12, m - 1
    x, g, w_t = np.zeros((m, k)), np.zeros((m, n)), np.zeros((k, n))
    x[at] = [2, 2, 1, 1] * 3                            # kept: the twos; s = 1.5, so every channel of R is +-1
    g[at, :3] = 1
    a, b = np.zeros((r, k)), np.zeros((n, r))
    for j, end, chans in ((0, 2.0 ** -20, (2, 3, 6)), (r - 1, -2.0 ** -20, (7, 10, 11))):
        b[:3, j] = 1, 2.0 ** -8, end
        a[j, list(chans)] = 1, 2.0 ** -8, end           # pruned channels only: D is zero, dX is U A
    kept = training.checkpoint(dev(x))
    assert np.array_equal(kept.unpack().double().cpu().numpy(), x)
    dx, da, db = training.sparse_linear_backward(dev(g), kept, dev(w_t), dev(a), dev(b))
    u = g @ b
    pruned = np.tile([0, 0, 1, 1], 3)
    rest = x[at] * (1 - 1.5 * (1 - pruned))
    for got, want in ((da, np.outer(u[at], rest)), (db, np.outer(g[at], rest @ a.T)),
                      (dx, np.where(np.arange(m)[:, None] == at, pruned * (u @ a), 0))):
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().bfloat16())


@pytest.mark.parametrize("m,k", [(1, 4), (7, 8), (40, 36), (41, 68), (40, 516), (21, 1028), (10, 12292)])
def test_statistics_of_rows_of_any_magnitude(m, k):
    """Rows of 2^-120 to 2^100, half-zero rows and subnormal ones: s and Lk are sums
    of positive fp32 numbers (subnormals are kept, so there is no absolute term)."""
    print("[statistics]", m, k, file=sys.stderr, flush=True)
    bits = gen.uniform_bits(np.random.default_rng(m + k), (m, k), emax=100, span=220)
    bits[::3, :k // 2] = 0
    bits[1::5] &= 0x807f
    bits[2::7, 1:] = 0                                             # one channel: s is 1
    x = to_dev(bits)
    kept = training.checkpoint(x)
    v, mk = plain.bf16(x), plain.mask(kept.idx.cpu().numpy(), k)
    lk, l1 = (mk * np.abs(v)).sum(1), np.abs(v).sum(1)
    s, got = np.where(lk > 0, l1 / np.where(lk > 0, lk, 1), 1), kept.stats.cpu().double().numpy()
    tol = (k / 128 + 16) * plain.U24
    assert (np.abs(got[:, 1] - lk) <= tol * lk).all()
    assert (np.abs(got[:, 0] - s) <= 3 * tol * s).all()
    assert torch.equal(kept.stats[:, 0], rtl.sparsify_2of4(x)[2])  # the forward's scale, bit for bit


@pytest.mark.parametrize("law", ["mixture", "gelu", "ties"])
@pytest.mark.parametrize("m,n,k,r", [(64, 128, 256, 16), (33, 260, 516, 64), (5, 36, 68, 0)])
def test_the_layer_on_the_stored_values_is_the_layer(m, n, k, r, law):
    """y from the layer, and the fp64 layer on the stored values, positions and
    scales, agree to the checkpoint's error: half a step of every code through the
    products, and the layer's own roundings."""
    print("[layer]", m, n, k, r, law, file=sys.stderr, flush=True)
    rng, alpha = np.random.default_rng(m + n), 0.75
    x = to_dev({"mixture": gen.mixture_bernoulli, "gelu": gen.gelu_of_normal, "ties": gen.tie_heavy}[law](rng, m, k))
    w, a, b = (dev(std * rng.standard_normal(sh)) for sh, std in (((n, k), 0.05), ((r, k), 0.05), ((n, r), 0.05)))
    y = rtl.sparse_linear(x, w, a, b, alpha) if r else rtl.sparse_linear(x, w)
    kept = training.checkpoint(x)
    codes, exps = kept.codes.cpu().numpy(), kept.exps.cpu().numpy()
    v, mk, s = plain.values(codes, exps), plain.mask(kept.idx.cpu().numpy(), k), plain.bf16(kept.stats[:, :1])
    half = np.repeat(2.0 ** (exps.astype(np.float64) - 134), 32, 1)[:, :k]
    assert (np.abs(v - plain.bf16(x)) <= half).all()
    W, A, B = (plain.bf16(t) for t in (w, a, b))
    up = np.abs(A.T) @ np.abs(B.T) * abs(alpha)
    rest, scaled = v * (1 - s * mk), s * mk * v
    want = scaled @ W.T + alpha * rest @ A.T @ B.T
    reach, reach_r = np.abs(scaled) + s * mk * half, np.abs(rest) + np.abs(1 - s * mk) * half
    tol = (s * mk * half) @ np.abs(W.T) + (np.abs(1 - s * mk) * half) @ up
    tol += 2 * plain.depth(k) * plain.U24 * (reach @ np.abs(W.T)) + (2 * plain.depth(k) * plain.U24 + plain.U16) * (reach_r @ up)
    got = plain.bf16(y)
    assert (np.abs(got - want) <= tol + plain.HALF_BF16 * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("m,n,k,r", [(70, 136, 260, 16), (600, 264, 1032, 64), (33, 64, 68, 100), (70, 136, 260, 0)])
def test_what_a_gradient_that_is_not_finite_reaches(m, n, k, r, value):
    """Its token's row of dX, dA, and its channel's row of dB."""
    rng, row, col = np.random.default_rng(m), m // 2, n // 3
    x, g = to_dev(gen.mixture_bernoulli(rng, m, k)), dev(0.01 * rng.standard_normal((m, n)))
    w_t, a, b = (dev(0.05 * rng.standard_normal(s)) for s in ((k, n), (r, k), (n, r)))
    lora = (a, b) if r else (None, None)
    for fine in (False, True):
        kept = training.checkpoint(x, fine=fine)
        want = training.sparse_linear_backward(g, kept, w_t, *lora)
        bad = g.clone()
        bad[row, col] = value
        got = training.sparse_linear_backward(bad, kept, w_t, *lora)
        others = torch.arange(m, device=DEV) != row
        assert torch.equal(got[0][others], want[0][others]) and not bool(torch.isfinite(got[0][row]).any())
        if r:
            assert not bool(torch.isfinite(got[1]).any()) and not bool(torch.isfinite(got[2][col]).any())
            rest = torch.arange(n, device=DEV) != col
            assert torch.equal(got[2][rest], want[2][rest])
