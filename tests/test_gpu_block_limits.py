"""Offsets that pass 32 bits: long caches, many tokens; memory is given back."""
import gc

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention, norm  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def give_back():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def far_cache(n, heads, d, seed):
    """Zero keys and values but for one far row and one near one per head."""
    k, v = torch.zeros(n, heads, d, dtype=BF, device=DEV), torch.zeros(n, heads, d, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(seed)
    for at in (5, n - 3):
        k[at] = 4.0
        v[at] = torch.randn(heads, d, generator=g).to(BF).to(DEV)
    return k, v


def test_a_cache_past_4_gib():
    """Two keys with score 4 d / sqrt d = 45.25 among zeros: half of each one's value, to e^-45 n."""
    n, h, d = 2_200_000, 8, 128
    k, v = far_cache(n, h, d, 1)
    q = torch.ones(1, 1, h, d, dtype=BF, device=DEV)
    want = (v[5].double() + v[n - 3].double()) / 2
    for lens in (None, torch.tensor([n - 1], dtype=torch.int32, device=DEV)):
        o = attention.attention(q, k[None], v[None], k_lens=lens)[0, 0].double()
        assert ((o - want).abs() <= 2.0 ** -8 * (want.abs() + 1e-6) + 1e-6).all()
    many = q.expand(1, 200, h, d).contiguous()
    o = attention.attention(many, k[None], v[None])[0].double()
    assert ((o - want).abs() <= 2.0 ** -8 * (want.abs() + 1e-6) + 1e-6).all()


def test_packed_rows_past_4_gib():
    """A sequence at the far end of a tensor, forward and backward, as by itself; the rest is zero."""
    n, h, d = 2_200_000, 8, 128
    big = torch.zeros(n, h, d, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(2)
    q, k, v, do = ((torch.randn(150, h, d, generator=g)).to(BF).to(DEV) for _ in range(4))
    big[n - 150:] = k
    starts = torch.tensor([n - 150, n], dtype=torch.int32, device=DEV)
    own = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    want = attention.attention(q, k, v, causal=True, q_starts=own, return_lse=True)
    grads = attention.attention_backward(do, q, k, v, *want, causal=True, q_starts=own)
    values = torch.zeros_like(big)
    values[n - 150:] = v
    got = attention.attention(q, big, values, causal=True, q_starts=own, k_starts=starts, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dq, dk, dv = attention.attention_backward(do, q, big, values, *got, causal=True, q_starts=own, k_starts=starts)
    assert torch.equal(dq, grads[0]) and torch.equal(dk[n - 150:], grads[1]) and torch.equal(dv[n - 150:], grads[2])
    assert not dk[:n - 150].any() and not dv[:n - 150].any()


def test_norm_past_4_gib():
    n, c = 2_200_000, 1024
    x = torch.zeros(n, c, dtype=BF, device=DEV)
    x[-7:] = torch.randn(7, c, generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    y, m, r = norm.layer_norm(x, return_stats=True)
    want = norm.layer_norm(x[-7:], return_stats=True)
    assert torch.equal(y[-7:], want[0]) and torch.equal(m[-7:], want[1]) and not y[:-7].any()
    dx = norm.layer_norm_backward(x, x, m, r)[0]
    assert torch.equal(dx[-7:], norm.layer_norm_backward(x[-7:], x[-7:], *want[1:])[0])


def test_many_sequences():
    """More workgroups than a grid's first dimension may hold threads for."""
    b = 600_000
    q = torch.randn(b, 1, 8, 8, generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)
    o = attention.attention(q, q, q)
    assert torch.equal(o, q)
    q = q.view(b // 40, 40, 8, 8)
    lens = torch.ones(b // 40, dtype=torch.int32, device=DEV)
    assert torch.equal(attention.attention(q, q, q, k_lens=lens), q[:, :1].expand(-1, 40, -1, -1))
