"""Gradients where a query sees few keys: ds is a difference of near numbers there, and D must not carry o's
rounding.  The allowance counts the roundings of ds and of the results alone."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention as at  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_plain as plain  # noqa: E402
from test_gpu_attention import rand  # noqa: E402


@pytest.mark.parametrize("tk", [1, 2, 3, 17, 64, 65, 100, 128])
@pytest.mark.parametrize("tq", [1, 130, 300])
@pytest.mark.parametrize("d", [32, 128])
def test_few_keys(tq, tk, d):
    q, g = rand(1, tq, 4, d, seed=1), rand(1, tq, 4, d, seed=2)
    k, v = rand(1, tk, 2, d, seed=3), rand(1, tk, 2, d, seed=4)
    o, lse = at.attention(q, k, v, return_lse=True)
    dq, dk, dv = at.attention_backward(g, q, k, v, o, lse)
    for j in range(2):
        sums = [0, 0, 0, 0]
        for h in (2 * j, 2 * j + 1):
            r = plain.one(q[0, :, h], k[0, :, j], v[0, :, j], d ** -0.5, False, g[0, :, h], few=True)
            plain.check(dq[0, :, h], *r["dq"], f"dq of head {h}")
            sums = [a + b for a, b in zip(sums, (*r["dk"], *r["dv"]))]
        plain.check(dk[0, :, j], *sums[:2], f"dk of head {j}")
        plain.check(dv[0, :, j], *sums[2:], f"dv of head {j}")


def test_the_first_queries_of_a_causal_sequence():
    n, d = 90, 64
    q, k, v, g = (rand(n, 1, d, seed=i) for i in range(4))
    starts = torch.tensor([0, n], dtype=torch.int32, device=q.device)
    o, lse = at.attention(q, k, v, causal=True, q_starts=starts, return_lse=True)
    dq, dk, dv = at.attention_backward(g, q, k, v, o, lse, causal=True, q_starts=starts)
    r = plain.one(q[:, 0], k[:, 0], v[:, 0], d ** -0.5, True, g[:, 0], few=True)
    for got, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        plain.check(got[:, 0], *r[name], name)
