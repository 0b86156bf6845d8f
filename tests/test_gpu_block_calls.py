"""Calls of the block's operators that the documentation allows and no other test makes."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention as at, dense, norm  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


def rand(*shape, seed, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def test_attention_warns():
    q = rand(1, 4, 2, 16, seed=1).requires_grad_()
    with pytest.warns(UserWarning, match=r"attention\.attention records no autograd graph"):
        at.attention(q, q.detach(), q.detach())
    with torch.no_grad():
        assert not at.attention(q, q, q).requires_grad


def test_one_tensor_as_queries_keys_and_values():
    x, g = rand(2, 150, 4, 64, seed=2), rand(2, 150, 4, 64, seed=3)
    y, z = x.clone(), x.clone()
    got, want = at.attention(x, x, x, return_lse=True), at.attention(x, y, z, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for a, b in zip(at.attention_backward(g, x, x, x, *got), at.attention_backward(g, x, y, z, *want)):
        assert torch.equal(a, b)
    for a, b in zip(at.attention_backward(x, x, x, x, *got), at.attention_backward(y, x, y, z, *got)):
        assert torch.equal(a, b)


def test_rows_of_a_slice():
    """72 channels in rows of 240, 8-byte aligned; each of the two results is within half a step (2^-8) of the exact one."""
    x = rand(5, 33, 240, seed=4)[:, :, 100:172]
    w, b = rand(5, 72, seed=5), rand(5, 72, seed=6)
    y, m, r = norm.layer_norm(x, w, b, return_stats=True)
    want = norm.layer_norm(x.contiguous(), w, b, return_stats=True)
    for a, c in zip((y, m, r), want):
        assert torch.equal(a, c) or (a.double() - c.double()).abs().max() <= 2.0 ** -8 * c.double().abs().max()
    dy = rand(5, 33, 72, seed=7)
    got = norm.layer_norm_backward(dy, x, m, r, w)
    ref = norm.layer_norm_backward(dy, x.contiguous(), m, r, w)
    for a, c in zip(got, ref):
        assert (a.double() - c.double()).abs().max() <= 2.0 ** -8 * c.double().abs().max()


def test_a_gated_step_replayed():
    x, w, dy = rand(2, 40, 96, seed=8), rand(264, 96, seed=9), rand(2, 40, 264, seed=10)
    gate, res = rand(2, 264, seed=11), rand(2, 40, 264, seed=12)

    def step():
        y, z = dense.linear(x, w, activation="gelu", gate=gate, residual=res, keep=True)
        return (y, *dense.linear_backward(dy, x, w, z, activation="gelu", gate=gate))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(rand(2, 40, 96, seed=20 + i))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


@pytest.mark.parametrize("m", [16, 17, 31])
def test_few_rows_into_the_residual(m):
    x, w, res = rand(m, 4096, seed=13), rand(12000, 4096, seed=14) * 0.01, rand(m, 12000, seed=15)
    want = dense.linear(x, w, residual=res)
    assert torch.equal(dense.linear(x, w, residual=res, out=res), want)
    assert dense.linear(x[0], w).shape == (12000,)
