"""Strides of dimensions of one: whatever they are, no address depends on them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention as at  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF)


def test_one_token_of_a_large_batch_laid_out_tokens_first():
    """[1, batch, heads, d] transposed: its token stride, 9 million elements, is past what several tokens may have."""
    b, h, d = 1100, 64, 128
    x, k = rand(1, b, h, d, seed=1), rand(b, 2, 1, d, seed=2)
    q = x.transpose(0, 1)
    assert q.stride(1) >= 1 << 23
    want = at.attention(x[0][:, None].contiguous(), k, k, return_lse=True)
    out = torch.empty_like(x).transpose(0, 1)
    got = at.attention(q, k, k, out=out, return_lse=True)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    g = rand(b, 1, h, d, seed=3)
    grads = at.attention_backward(g, q, k, k, *got)
    assert all(torch.equal(a, c) for a, c in zip(grads, at.attention_backward(g, q.contiguous(), k, k, *want)))


def test_several_tokens_so_far_apart_are_refused():
    import activation_sparse_gemm_token_amd as rtl
    x = torch.zeros((1 << 23) + 64, dtype=BF, device=DEV)
    q = x.as_strided((1, 2, 1, 64), (0, 1 << 23, 64, 1))
    with pytest.raises(rtl.RtlError):
        at.attention(q, q, q)
