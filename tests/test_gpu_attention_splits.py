"""Attention where the work is split and joined: the last tiles of a batch over ranges of keys, and dK and
dV over ranges of queries."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention as at  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_attention import BF, HF, run_batch, run_packed  # noqa: E402


def meta(*s):
    return torch.empty(*s, dtype=BF, device="meta")


@pytest.mark.parametrize("b,tq,tk,hq,hk,d,dtype", [(1, 40, 600, 2, 1, 64, BF), (2, 300, 1030, 3, 3, 128, BF), (1, 129, 5000, 2, 2, 72, HF),
                                                   (1, 33, 513, 1, 1, 8, BF)])
def test_last_tiles_over_ranges_of_keys(b, tq, tk, hq, hk, d, dtype):
    assert at.workspace_bytes(meta(b, tq, hq, d), meta(b, tk, hk, d)) > 0
    assert at.workspace_bytes(meta(b, tq, hq, d), meta(b, tk, hk, d), causal=True) == 0
    run_batch(b, tq, tk, hq, hk, d, False, dtype=dtype)
    run_batch(b, tq, tk, hq, hk, d, True, dtype=dtype)
    run_batch(b, tq, tk, hq, hk, d, False, dtype=dtype, lens=[tk // 3, 0][:b])


def test_whole_rounds_and_the_rest():
    """More tiles than the card holds at a time, and some over."""
    b, tq, tk, h, d = 5, 1280, 768, 17, 96
    q, k = meta(b, tq, h, d), meta(b, tk, h, d)
    tiles = b * h * 10
    assert at.workspace_bytes(q, k) == 3 * (tiles - 768) * 128 * (d + 2) * 4 if tiles < 1536 else True
    run_batch(b, tq, tk, h, h, d, False)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("tq,tk,hq,hk,d", [(600, 600, 2, 1, 128), (1500, 70, 1, 1, 64), (300, 1000, 4, 1, 40), (513, 200, 2, 2, 96)])
def test_gradients_over_ranges_of_queries(tq, tk, hq, hk, d, causal):
    q, k = meta(1, tq, hq, d), meta(1, tk, hk, d)
    assert at.backward_workspace_bytes(q, k) >= 8 * tq * hq + 2 * 2 * tk * hk * d * 4
    run_batch(1, tq, tk, hq, hk, d, causal, back=True)
    run_batch(1, tq, tk, hq, hk, d, causal, lens=[tk // 2], back=True)
    run_packed([tq], [tk], hq, hk, d, causal, back=True, lead=3, tail=150)
    run_packed([tq, 0, 40], [tk, 5, 0], hq, hk, d, causal, back=True, lead=3, tail=150)
