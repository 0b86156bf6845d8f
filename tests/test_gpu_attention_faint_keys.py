"""One strong key and very many faint ones, whose weights are small each and not together: they count in both types.

The strong key's score is 0 and its value 0; n keys have the score -26 log 2 and the value 1: o = w / (1 + w) with w = n 2^-26,
and as much in every channel.  Allowed: the result's and the weights' half steps, and 2^-32 of the largest weight for a
weight in fp16 (half its smallest step, 2^-25, where the largest stands for 2^7).

The sum of the weights: a score is off by a few half steps of 26, which is the weight's relative error; a lane holds half
of its query's keys and adds 256 or 512 of them up, one at a time, before it adds them to its sum: at most 512 additions
beside the strong key, and n / 512 of parts, off by 2^-24 of the whole each.  That error, relative to 1 + w, goes into o
by as much of o and into the log-sum-exp as it is."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention as at  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("bits", [20, 26, 28])
@pytest.mark.parametrize("strong", ["first", "last", "middle"])
@pytest.mark.parametrize("tq,packed", [(1, False), (24, False), (40, False), (200, False), (40, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_faint_keys(dtype, tq, packed, strong, bits):
    n, d, heads = 400_000, 16, 2
    q = torch.ones(tq, heads, d, dtype=dtype, device=DEV)
    k = torch.full((n + 1, heads, d), -bits / 16.0, dtype=dtype, device=DEV)       # a score of -bits, times log 2
    v = torch.ones(n + 1, heads, d, dtype=dtype, device=DEV)
    at_ = {"first": 0, "last": n, "middle": n // 2}[strong]
    k[at_] = 0
    v[at_] = 0
    if packed:
        starts = [torch.tensor([0, m], dtype=torch.int32, device=DEV) for m in (tq, n + 1)]
        o, lse = at.attention(q, k, v, scale=math.log(2), q_starts=starts[0], k_starts=starts[1], return_lse=True)
    else:
        o, lse = (t[0] for t in at.attention(q[None], k[None], v[None], scale=math.log(2), return_lse=True))
    w = n * 2.0 ** -bits
    h = torch.finfo(dtype).eps / 2
    tiny = n * 2.0 ** -32 if dtype is torch.float16 else 0.0
    sums = (4 * bits + 64 + 512 + n / 512) * 2.0 ** -24
    assert ((o.double() - w / (1 + w)).abs() <= (2 * h * 1.01 + sums) * w / (1 + w) + tiny).all()
    assert ((lse.double() - math.log1p(w)).abs() <= sums).all()
