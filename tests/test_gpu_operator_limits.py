"""The operators beside the layer at the largest sizes that their headers admit."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import training  # noqa: E402

DEV = "cuda:0"


def say(*a):
    print("[limits]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("m,k", [((1 << 26) - 3, 4), (1 << 26, 4), ((1 << 26) + 5, 12), ((1 << 28) - 257, 4)])
def test_checkpoint_of_the_most_tokens(m, k):
    """More workgroups than one launch dimension holds threads for."""
    say(m, k)
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(m, device=DEV)
    x[:, 0] = (at % 113 + 1).bfloat16()                            # exact
    x[:, 2] = -1
    kept = training.checkpoint(x)
    first, exps = x[:, 0].float(), kept.exps[:, 0].int()
    right = {"scale": kept.stats[:, 0] == 1, "kept": kept.stats[:, 1] == first + 1,
             "exponent": (torch.ldexp(torch.ones_like(first), exps - 127) <= first) &
                         (torch.ldexp(torch.ones_like(first), exps - 126) > first),
             "positions": (kept.idx[:, 0] & 15) == 0 + (2 << 2), "values": kept.unpack() == x}
    wrong = [n for n, ok in right.items() if not bool(ok.all())]   # names only: a failure prints no tensor of this size
    assert wrong == []
