"""Queries and keys rotated in place inside a fused projection's output, whatever
the order of its dimensions in memory."""
import itertools
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import rotary  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("order", list(itertools.permutations(range(3))) + ["beside"])
@pytest.mark.parametrize("b,t,hq,hk,d,layout", [(2, 33, 6, 2, 64, "half"), (3, 7, 2, 2, 40, "interleaved"), (1, 1, 4, 4, 6, "half")])
def test_in_place_in_any_order(order, b, t, hq, hk, d, layout):
    print("[rotary]", order, b, t, hq, hk, d, layout, file=sys.stderr, flush=True)
    g = torch.Generator().manual_seed(t)
    if order == "beside":                                          # [batch, tokens, heads, (q, k, v), channels]
        x = torch.randn(b, t, hq, 3, d, generator=g).bfloat16().to(DEV)
        q, k, v = x[:, :, :, 0], x[:, :, :, 1], x[:, :, :, 2]
    else:
        shape = [(b, t, hq + 2 * hk)[i] for i in order]
        x = torch.randn(*shape, d, generator=g).bfloat16().to(DEV)
        y = x.permute(*[order.index(i) for i in range(3)], 3)
        q, k, v = y[:, :, :hq], y[:, :, hq:hq + hk], y[:, :, hq + hk:]
    pos = torch.arange(t, device=DEV) + 1000
    freq = rotary.frequencies(d if d > 6 else 4).to(DEV)
    want, kept = rotary.rope(q, pos, freq, k=k, layout=layout), v.clone()
    out = rotary.rope(q, pos, freq, k=k, layout=layout, out=q, k_out=k)
    assert out[0] is q and out[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)
