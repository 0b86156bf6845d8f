"""Packed batches of more sequences than a wavefront has lanes: a workgroup finds its own by a search, so that their number
adds no walk to each.  A sequence's results have the same bits in any packed batch."""
import gc
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention as at  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def give_back():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def rand(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


def lengths(n, most, seed):
    """Sequences of 0 to `most` tokens, with a few long ones and tile ends among them."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, most + 1, (n,), generator=g)
    lens[0], lens[n // 3], lens[n // 2], lens[n - 2] = 128, 700, 257, 127
    lens[n // 5:n // 5 + 4] = 0
    return lens.tolist()


def starts_of(lens, lead):
    return [lead + s for s in (0, *torch.tensor(lens).cumsum(0).tolist())]


def on_device(starts):
    return torch.tensor(starts, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("other_keys", [False, True])
@pytest.mark.parametrize("n", [65, 66, 129, 1000, 4095, 4096, 4097])
def test_as_in_batches_of_few(n, other_keys):
    """All at once, and 60 sequences at a time."""
    hq, hk, d, causal = 2, 1, 32, n % 2 == 0
    lq = lengths(n, 40 if n > 1000 else 90, n)
    lk = lengths(n, 60, n + 1) if other_keys else lq
    qs, ks = starts_of(lq, 3), starts_of(lk, 7 if other_keys else 3)
    nq, nk = qs[-1] + 300, ks[-1] + 5 if other_keys else qs[-1] + 300
    q, g, k, v = rand(nq, hq, d, seed=1), rand(nq, hq, d, seed=2), rand(nk, hk, d, seed=3), rand(nk, hk, d, seed=4)
    args = dict(causal=causal, q_starts=on_device(qs), k_starts=on_device(ks))
    o, lse = at.attention(q, k, v, return_lse=True, **args)
    grads = at.attention_backward(g, q, k, v, o, lse, **args)
    for i in range(0, n, 60):
        a, b = qs[i], qs[min(i + 60, n)]
        c, e = ks[i], ks[min(i + 60, n)]
        part = dict(causal=causal, q_starts=on_device([s - a for s in qs[i:i + 61]]), k_starts=on_device([s - c for s in ks[i:i + 61]]))
        po, pl = at.attention(q[a:b], k[c:e], v[c:e], return_lse=True, **part)
        assert torch.equal(o[a:b], po) and torch.equal(lse[:, a:b], pl), i
        dq, dk, dv = at.attention_backward(g[a:b], q[a:b], k[c:e], v[c:e], po, pl, **part)
        assert torch.equal(grads[0][a:b], dq) and torch.equal(grads[1][c:e], dk) and torch.equal(grads[2][c:e], dv), i
    for t, first, last in ((o, qs[0], qs[-1]), (grads[0], qs[0], qs[-1]), (grads[1], ks[0], ks[-1]), (grads[2], ks[0], ks[-1])):
        assert not t[:first].any() and not t[last:].any()
    assert (lse[:, :qs[0]] == -math.inf).all() and (lse[:, qs[-1]:] == -math.inf).all()


def test_many_tokens_alone():
    """300 000 sequences of one token: the value itself, in every head that shares it."""
    n, hq, hk, d = 300_000, 8, 2, 16
    q, k, v, g = (rand(n, h, d, seed=i) for i, h in enumerate((hq, hk, hk, hq)))
    starts = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    o, lse = at.attention(q, k, v, q_starts=starts, return_lse=True)
    assert torch.equal(o, v.repeat_interleave(hq // hk, 1))
    s = (q.double() * k.double().repeat_interleave(hq // hk, 1)).sum(-1) * d ** -0.5
    size = (q.double().abs() * k.double().abs().repeat_interleave(hq // hk, 1)).sum(-1) * d ** -0.5
    assert ((lse.double() - s.t()).abs() <= (d + 16) * 2.0 ** -24 * size.t()).all()
    dv = at.attention_backward(g, q, k, v, o, lse, q_starts=starts)[2]
    want = g.double().view(n, hk, hq // hk, d).sum(2)
    size = g.double().abs().view(n, hk, hq // hk, d).sum(2)
    # p is 1 to its exponent's error, rounded to 1; four summands, then the result's half step.
    assert ((dv.double() - want).abs() <= 2.0 ** -8 * want.abs() + 8 * 2.0 ** -24 * size).all()


def test_a_million_sequences():
    """Of 0, 1 or 2 tokens, causal: the first token's result is its value, the second's lies between both."""
    n, d = 1_000_000, 8
    lens = torch.randint(0, 3, (n,), generator=torch.Generator(device=DEV).manual_seed(9), device=DEV)
    starts = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).int()
    total = int(starts[-1])
    q, k, v = (rand(total, 4, d, seed=i) for i in range(3))
    o = at.attention(q, k, v, causal=True, q_starts=starts)
    first = starts[:-1][lens > 0].long()
    assert torch.equal(o[first], v[first])
    one = starts[:-1][lens == 2].long()
    s = torch.stack([(q[one + 1].double() * k[one + j].double()).sum(-1) for j in (0, 1)], -1) * d ** -0.5
    p = torch.softmax(s, -1)
    want = p[..., :1] * v[one].double() + p[..., 1:] * v[one + 1].double()
    size = p[..., :1] * v[one].double().abs() + p[..., 1:] * v[one + 1].double().abs()
    # Weights rounded to bf16 and the result too, half a step each; fp32's few steps of scores below 64.
    assert ((o[one + 1].double() - want).abs() <= 2.0 ** -8 * (want.abs() + size) * 1.01 + 64 * 40 * 2.0 ** -24 * size).all()
