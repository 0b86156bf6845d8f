"""The operators beside the layer at the largest sizes that their headers admit."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import rotary, training, w4  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def give_back():
    """These hold up to half of the card: nothing of it stays in torch's cache."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


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
             "exponent": torch.frexp(first).exponent == exps - 126,
             "positions": (kept.idx[:, 0] & 15) == 0 + (2 << 2), "values": kept.unpack() == x}
    wrong = [n for n, ok in right.items() if not bool(ok.all())]   # names only: a failure prints no tensor of this size
    assert wrong == []


@pytest.mark.parametrize("m,n", [(1, (1 << 28) + 17), (17, (1 << 29) + 33)])
def test_4_bit_weight_of_the_most_rows(m, n):
    """The same of w4.linear: short channels, and the form for more rows."""
    say(m, n)
    g = torch.Generator(device=DEV).manual_seed(m)
    k = 32
    x = torch.randint(-3, 4, (m, k), generator=g, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(1, 5, (n, 1), generator=g, device=DEV).bfloat16() / 4
    y = w4.linear(x, w4.pack(codes, scales, group=32))
    step = 1 << 22
    wrong = 0
    for lo in list(range(0, n, 17 * step)) + [n - step]:           # parts of it, its end among them
        part = codes[lo:lo + step]
        q = torch.stack([part & 15, part >> 4], -1).flatten(1).float() - 8
        want = (x.float() @ q.t()) * scales[lo:lo + step, 0].float()    # whole quarters: exact in fp32
        wrong += int((y[:, lo:lo + step] != want.bfloat16()).sum())
    assert wrong == 0


def test_rotary_of_more_workgroups_than_a_launch_dimension():
    """2^26 tokens of 1024 channels (137 GB), four to a workgroup, in place."""
    t, d, first = (1 << 26) + 6, 1024, 1 << 20
    if torch.cuda.mem_get_info()[0] < (150 << 30):
        pytest.skip("needs 150 GB of free device memory")
    x = torch.empty(t, 1, d, dtype=torch.bfloat16, device=DEV)
    x[:first] = torch.randn(first, 1, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).bfloat16()
    for lo in range(first, t, first):                              # the same rows again and again
        x[lo:lo + first] = x[:min(first, t - lo)]
    pos = torch.arange(t, device=DEV) % 1021
    f = rotary.frequencies(d).to(DEV)
    head = x[:first].clone()
    rotary.rope(x, pos, f, out=x)
    bad = 0
    for lo in [0, first, 31 * first, (1 << 24) * 4 - 4 - first, t // first * first]:
        n = min(first, t - lo)
        row = torch.arange(lo, lo + n, device=DEV) % first
        bad += int((x[lo:lo + n] != rotary.rope(head[row], pos[lo:lo + n].contiguous(), f)).sum())
    assert bad == 0
