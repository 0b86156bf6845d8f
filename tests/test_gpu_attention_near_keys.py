"""Gradients of queries that see few keys in a tile of 128 queries whose last ones see more: D is formed from p and dP for
each query that sees up to 128 keys, not for whole tiles, so o's rounding does not weigh on its dQ."""
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

DEV = "cuda:0"
BF = torch.bfloat16


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)


# (queries, keys): the last key's query is the last one, so query i sees i + 1 + keys - queries.
SIZES = [(300, 173), (300, 174), (300, 172), (256, 130), (129, 140), (200, 201), (128, 191), (128, 192), (131, 320), (513, 200), (140, 13),
         (700, 640)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("d", [32, 72, 128])
@pytest.mark.parametrize("nq,nk", SIZES)
def test_near_keys(nq, nk, d, packed):
    hq, hk = 2, 1
    q, k, v, g = rand(nq, hq, d, seed=1), rand(nk, hk, d, seed=2), rand(nk, hk, d, seed=3), rand(nq, hq, d, seed=4)
    if packed:
        args = dict(causal=True, q_starts=torch.tensor([0, nq], dtype=torch.int32, device=DEV),
                    k_starts=torch.tensor([0, nk], dtype=torch.int32, device=DEV))
        o, lse = at.attention(q, k, v, return_lse=True, **args)
        grads = at.attention_backward(g, q, k, v, o, lse, **args)
    else:
        o, lse = at.attention(q[None], k[None], v[None], causal=True, return_lse=True)
        grads = [t[0] for t in at.attention_backward(g[None], q[None], k[None], v[None], o, lse, causal=True)]
        o, lse = o[0], lse[0]
    plain.check_all(q, k, v, [(0, nq, 0, nk)], d ** -0.5, True, o, lse, g, grads)
    seen = torch.arange(nq, device=DEV) + 1 + nk - nq
    near = seen <= 128
    for h in range(hq):
        want, allow = plain.one(q[:, h], k[:, 0], v[:, 0], d ** -0.5, True, g[:, h], few=True)["dq"]
        plain.check(grads[0][near, h], want[near], allow[near], f"dq of head {h}")


def test_a_cache_of_near_keys():
    """Filled lengths that put the same boundary into a batch's tiles."""
    b, tq, tk, d = 4, 260, 300, 64
    q, k, v, g = rand(b, tq, 1, d, seed=5), rand(b, tk, 1, d, seed=6), rand(b, tk, 1, d, seed=7), rand(b, tq, 1, d, seed=8)
    lens = [133, 2, 262, 300]
    k_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, lse = at.attention(q, k, v, causal=True, k_lens=k_lens, return_lse=True)
    dq, dk, dv = at.attention_backward(g, q, k, v, o, lse, causal=True, k_lens=k_lens)
    for i, n in enumerate(lens):
        near = torch.arange(tq, device=DEV) + 1 + n - tq <= 128
        r = plain.one(q[i, :, 0], k[i, :n, 0], v[i, :n, 0], d ** -0.5, True, g[i, :, 0], few=True)
        plain.check(dq[i, near, 0], r["dq"][0][near], r["dq"][1][near], f"dq of sequence {i}")
        assert (dk[i, n:] == 0).all() and (dv[i, n:] == 0).all()
