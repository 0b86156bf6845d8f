"""How exact the training calls are: what is carried between the products, the
checkpoint's own error in the gradients, and its statistics."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import training  # noqa: E402

DEV = "cuda:0"


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
