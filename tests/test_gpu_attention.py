"""Attention against fp64, with tolerances from the roundings on the way (attn_plain.py)."""
import math
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
BF, HF = torch.bfloat16, torch.float16


def rand(*shape, seed, dtype=BF, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def flat(t):
    """A batch's tensor as one packed one."""
    return t.reshape(-1, *t.shape[2:])


def flat_lse(lse):
    return lse.transpose(0, 1).reshape(lse.shape[1], -1)


def run_batch(b, tq, tk, hq, hk, d, causal, dtype=BF, lens=None, back=False, scale=None, seed=0, std=1.0):
    q, k, v = rand(b, tq, hq, d, seed=seed, dtype=dtype, std=std), rand(b, tk, hk, d, seed=seed + 1, dtype=dtype), \
        rand(b, tk, hk, d, seed=seed + 2, dtype=dtype)
    k_lens = None
    if lens is not None:
        k_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        for i, n in enumerate(lens):                               # behind the filled rows: anything
            k[i, max(n, 0):] = math.nan
            v[i, max(n, 0):] = math.inf
    o, lse = at.attention(q, k, v, causal=causal, scale=scale, k_lens=k_lens, return_lse=True)
    g = grads = None
    if back:
        g = rand(b, tq, hq, d, seed=seed + 3, std=0.5)
        grads = at.attention_backward(g, q, k, v, o, lse, causal=causal, scale=scale, k_lens=k_lens)
    n = [tk] * b if lens is None else [min(max(i, 0), tk) for i in lens]
    spans = [(i * tq, (i + 1) * tq, i * tk, i * tk + n[i]) for i in range(b)]
    plain.check_all(flat(q), flat(k), flat(v), spans, d ** -0.5 if scale is None else scale, causal, flat(o), flat_lse(lse),
                    None if g is None else flat(g), None if grads is None else [flat(t) for t in grads])
    if back and lens is not None:
        for i in range(b):
            assert (grads[1][i, n[i]:] == 0).all() and (grads[2][i, n[i]:] == 0).all()
    return o, lse, grads


def run_packed(lens_q, lens_k, hq, hk, d, causal, dtype=BF, back=False, lead=0, tail=0, seed=0):
    """Sequences one after another, `lead` and `tail` rows of NaN around them."""
    nq, nk = lead + sum(lens_q) + tail, lead + sum(lens_k) + tail
    q, k, v = rand(nq, hq, d, seed=seed, dtype=dtype), rand(nk, hk, d, seed=seed + 1, dtype=dtype), \
        rand(nk, hk, d, seed=seed + 2, dtype=dtype)
    g = rand(nq, hq, d, seed=seed + 3, std=0.5)
    for t, n in ((q, nq), (k, nk), (v, nk), (g, nq)):
        t[:lead] = math.nan
        t[n - tail:] = math.nan
    starts = [torch.tensor([lead + sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=DEV)
              for n in (lens_q, lens_k)]
    same = lens_q == lens_k
    args = dict(causal=causal, q_starts=starts[0], k_starts=None if same else starts[1])
    o, lse = at.attention(q, k, v, return_lse=True, **args)
    grads = at.attention_backward(g, q, k, v, o, lse, **args) if back else None
    spans = [(a, b, c, e) for a, b, c, e in zip(*(s.tolist()[i:][:len(lens_q)] for s in starts for i in (0, 1)))]
    plain.check_all(q, k, v, spans, d ** -0.5, causal, o, lse, g if back else None, grads)
    for t, n in ((o, nq), *(((grads[0], nq), (grads[1], nk), (grads[2], nk)) if back else ())):
        assert (t[:lead] == 0).all() and (t[n - tail:] == 0).all()
    if lead or tail:
        assert (lse[:, :lead] == -math.inf).all() and (lse[:, nq - tail:] == -math.inf).all()
    return o, lse, grads


LENGTHS = [(1, 1), (1, 77), (3, 2), (5, 3), (31, 33), (64, 64), (65, 129), (127, 200), (128, 128), (130, 62), (257, 300)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("tq,tk", LENGTHS)
def test_packed_lengths(tq, tk, causal):
    """One sequence, alone in its tensor: the kernels for whole sequences, forward and backward."""
    run_packed([tq], [tk], 2, 1, 64, causal, back=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("tq,tk", LENGTHS)
def test_batch_lengths(tq, tk, causal):
    """The kernel for few queries, and the backward pass of a batch."""
    run_batch(2, tq, tk, 2, 1, 64, causal, back=True)


@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 64, 72, 88, 96, 104, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_head_dims(d, dtype):
    run_packed([70, 133], [70, 133], 3, 3, d, True, dtype=dtype, back=dtype is BF)
    run_batch(2, 40, 90, 3, 3, d, False, dtype=dtype, back=dtype is BF)


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (6, 2), (8, 8), (7, 1), (12, 4)])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_heads(hq, hk, causal):
    run_packed([50, 131], [50, 131], hq, hk, 72, causal, back=True)
    run_batch(2, 3, 700, hq, hk, 128, causal)
    run_batch(1, 40, 70, hq, hk, 64, causal, back=True)


@pytest.mark.parametrize("causal", [False, True])
def test_packed_ragged(causal):
    """Empty sequences, one token, ends inside tiles, NaN before the first and behind the last."""
    lens = [0, 1, 63, 64, 65, 0, 128, 129, 200, 1, 0]
    run_packed(lens, lens, 4, 2, 64, causal, back=True, lead=5, tail=37)
    other = [3, 0, 70, 64, 1, 5, 300, 2, 129, 40, 0]
    run_packed(lens, other, 2, 2, 96, causal, back=True, lead=2, tail=200)


def test_many_short_sequences():
    """More sequences than lanes that look for theirs."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 9, (150,), generator=g).tolist()
    run_packed(lens, lens, 2, 1, 32, True, back=True, tail=3)


@pytest.mark.parametrize("causal", [False, True])
def test_filled_lengths(causal):
    """A cache's filled rows: none, some, all, more than there are; what lies behind is never used."""
    run_batch(6, 5, 200, 4, 2, 64, causal, lens=[0, 1, 4, 129, 200, 300], back=True)
    run_batch(4, 1, 3000, 4, 2, 128, causal, lens=[2999, 17, 0, 3000])
    run_batch(3, 150, 300, 2, 2, 64, causal, lens=[20, 300, -5], back=True)


@pytest.mark.parametrize("causal", [False, True])
def test_batch_of_many_heads(causal):
    """Enough tiles for the kernel for whole sequences on a batch, some of them cut."""
    run_batch(18, 150, 170, 8, 4, 64, causal, lens=[170 - 9 * i for i in range(18)], back=True)


@pytest.mark.parametrize("tq,tk,hq,hk,d", [(1, 16385, 8, 1, 128), (1, 40001, 2, 2, 64), (7, 5000, 4, 2, 40), (33, 2050, 3, 1, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_queries_over_many_keys(tq, tk, hq, hk, d, dtype):
    """Keys split over workgroups and joined."""
    q = torch.empty(2, tq, hq, d, dtype=dtype, device="meta")
    assert at.workspace_bytes(q, torch.empty(2, tk, hk, d, device="meta")) > 0
    run_batch(2, tq, tk, hq, hk, d, True, dtype=dtype)
    run_batch(2, tq, tk, hq, hk, d, True, dtype=dtype, lens=[tk - 1, tk // 9])


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0, 4.0])
def test_scales(scale):
    """From even weights to a softmax that is one key's; the maximum moves often."""
    run_batch(1, 70, 300, 2, 2, 64, False, scale=scale, back=True)
    run_batch(1, 1, 4000, 2, 1, 64, False, scale=scale)


@pytest.mark.parametrize("packed", [False, True])
def test_rising_scores(packed):
    """Every step's scores pass the maximum before them; the largest is last."""
    n, d = 400, 64
    q = torch.ones(n, 1, d, dtype=BF, device=DEV)
    k = (torch.arange(n, device=DEV)[:, None, None] / 8).expand(n, 1, d).to(BF).contiguous()
    v = rand(n, 1, d, seed=3)
    if packed:
        starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        o, lse = at.attention(q, k, v, q_starts=starts, return_lse=True)
    else:
        o, lse = (t[0] for t in at.attention(q[None], k[None], v[None], return_lse=True))
    plain.check_all(q, k, v, [(0, n, 0, n)], d ** -0.5, False, o, lse)


def test_strides():
    """Slices of a fused projection, heads before tokens, a key that all queries' heads and tokens share."""
    qkv = rand(2, 90, 4 + 2 + 2, 64, seed=1)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    want = at.attention(q.contiguous(), k.contiguous(), v.contiguous(), return_lse=True)
    got = at.attention(q, k, v, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    heads_first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    assert torch.equal(at.attention(*heads_first), want[0])
    g = rand(2, 90, 4, 64, seed=2)
    grads = at.attention_backward(g, q, k, v, *want)
    again = at.attention_backward(g.transpose(1, 2).contiguous().transpose(1, 2), *heads_first, *want)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    one = rand(1, 1, 2, 64, seed=4).expand(2, 90, 2, 64)
    assert torch.equal(at.attention(q, one, one), at.attention(q, one.contiguous(), one.contiguous()))
    out = torch.full((2, 90, 6, 64), 7.0, dtype=BF, device=DEV)
    res = at.attention(q, k, v, out=out[:, :, 1:5])
    assert res.data_ptr() == out[:, :, 1:5].data_ptr() and torch.equal(res, want[0])
    assert (out[:, :, 0] == 7).all() and (out[:, :, 5] == 7).all()


def test_rows_in_no_sequence_of_a_given_output():
    q, k, v = (rand(100, 2, 64, seed=i) for i in range(3))
    starts = torch.tensor([4, 20, 20, 90], dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 3.0)
    at.attention(q, k, v, q_starts=starts, out=out)
    assert (out[:4] == 3).all() and (out[90:] == 3).all()
    new = at.attention(q, k, v, q_starts=starts)
    assert torch.equal(new[4:90], out[4:90]) and (new[:4] == 0).all() and (new[90:] == 0).all()


def test_starts_outside_the_tensor_are_cut():
    q, k, v = (rand(60, 2, 64, seed=i) for i in range(3))
    starts = lambda *n: torch.tensor(n, dtype=torch.int32, device=DEV)  # noqa: E731
    got = at.attention(q, k, v, q_starts=starts(-7, 20, 10, 900))
    assert torch.isfinite(got).all()
    want = at.attention(q, k, v, q_starts=starts(0, 20, 60))
    assert torch.equal(got[:10], want[:10])
    assert torch.equal(at.attention(q, k, v, q_starts=starts(0, 60, 5000)), at.attention(q, k, v, q_starts=starts(0, 60)))


def test_empty_calls():
    e = lambda *s: torch.empty(*s, dtype=BF, device=DEV)  # noqa: E731
    assert at.attention(e(0, 5, 2, 64), e(0, 7, 2, 64), e(0, 7, 2, 64)).shape == (0, 5, 2, 64)
    assert at.attention(e(2, 0, 2, 64), e(2, 7, 2, 64), e(2, 7, 2, 64)).shape == (2, 0, 2, 64)
    o, lse = at.attention(rand(2, 5, 2, 64, seed=1), e(2, 0, 2, 64), e(2, 0, 2, 64), return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = rand(6, 2, 64, seed=1)
    o, lse = at.attention(x, x, x, q_starts=none, return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert all((t == 0).all() for t in at.attention_backward(x, x, x, x, o, lse, q_starts=none))
    q = rand(2, 5, 2, 64, seed=1)
    o, lse = at.attention(q, e(2, 0, 2, 64), e(2, 0, 2, 64), return_lse=True)
    dq, dk, dv = at.attention_backward(q, q, e(2, 0, 2, 64), e(2, 0, 2, 64), o, lse)
    assert (dq == 0).all() and dk.shape == (2, 0, 2, 64)
    k = rand(2, 9, 2, 64, seed=2)
    q0 = e(2, 0, 2, 64)
    dq, dk, dv = at.attention_backward(q0, q0, k, k, q0, torch.empty(2, 2, 0, device=DEV))
    assert (dk == 0).all() and (dv == 0).all() and dq.shape == q0.shape


def test_the_same_bits_again_and_captured():
    """Replays between eager calls; no sum's order changes."""
    q, k, v, g = (rand(2, 200, 4, 64, seed=i) for i in range(4))
    q1, cache = rand(2, 1, 4, 64, seed=9), rand(2, 4000, 2, 64, seed=10)

    def step():
        o, lse = at.attention(q, k, v, causal=True, return_lse=True)
        return (o, lse, *at.attention_backward(g, q, k, v, o, lse, causal=True), at.attention(q1, cache, cache))

    want = step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_gradient_against_differences():
    """Along one direction: the loss's own change, from fp64 on the same inputs."""
    q, k, v, g = (rand(1, 50, 2, 32, seed=i) for i in range(4))
    o, lse = at.attention(q, k, v, causal=True, return_lse=True)
    grads = at.attention_backward(g, q, k, v, o, lse, causal=True)
    dirs = [rand(1, 50, 2, 32, seed=20 + i).double() for i in range(3)]

    def loss(t):
        total = 0.0
        x = [a.double() + t * b for a, b in zip((q, k, v), dirs)]
        for h in range(2):
            s = torch.mm(x[0][0, :, h], x[1][0, :, h].t()) / math.sqrt(32)
            p = torch.softmax(s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(1), -math.inf), 1)
            total += float((torch.mm(p, x[2][0, :, h]) * g[0, :, h].double()).sum())
        return total

    numeric = (loss(1e-5) - loss(-1e-5)) / 2e-5
    mine = sum(float((a.double() * b).sum()) for a, b in zip(grads, dirs))
    # Each of the 9600 terms is off by 3 bf16 half steps of its magnitude at most, in either direction.
    size = math.sqrt(sum(float(((a.double() * b) ** 2).sum()) for a, b in zip(grads, dirs)))
    assert abs(mine - numeric) <= 4 * 3 * 2.0 ** -8 * size
