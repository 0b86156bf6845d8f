"""Calls that record no autograd graph say so where a gradient would get lost."""
import warnings

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import layers, rotary, training, w4  # noqa: E402

DEV = "cuda:0"


def rand(*s):
    return (0.1 * torch.randn(*s, device=DEV)).bfloat16()


def calls():
    x, w, a, b = rand(8, 64), rand(32, 64), rand(4, 64), rand(32, 4)
    policy = layers.LayerPolicy(2, dense=[1])
    weight = w4.pack(torch.zeros(16, 32, dtype=torch.uint8, device=DEV), torch.ones(16, 2, device=DEV).bfloat16(), group=32)
    q, k, pos, f = rand(8, 2, 32), rand(8, 1, 32), torch.arange(8, device=DEV), rotary.frequencies(32).to(DEV)
    return {
        "sparse_linear": (lambda x, a, b: rtl.sparse_linear(x, w, a, b), [x, a, b]),
        "sparse_linear_noalloc": (lambda x, a, b: rtl.sparse_linear_noalloc(x, w, a, b), [x, a, b]),
        "prepare": (lambda x, a: rtl.apply(rtl.prepare(x, a), w, b), [x, a]),
        "apply": (lambda b: rtl.apply(rtl.prepare(x, a), w, b), [b]),
        "LayerPolicy.linear": (lambda x, a, b: policy.linear(0, x, w, a, b), [x, a, b]),
        "w4.linear": (lambda x: w4.linear(x, weight), [x]),
        "rotary.rope": (lambda q, k: torch.cat(rotary.rope(q, pos, f, k=k), 1), [q, k]),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_a_lost_gradient_is_named(name):
    call, args = calls()[name]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        want = call(*args)                                         # nothing requires a gradient
    for i in range(len(args)):
        mine = [t.detach().requires_grad_(j == i) for j, t in enumerate(args)]
        with pytest.warns(UserWarning, match=name.replace(".", r"\.") + " records no autograd graph") as seen:
            got = call(*mine)
        assert torch.equal(got, want) and not got.requires_grad
        assert seen[0].filename == __file__                        # the caller's line
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                assert torch.equal(call(*mine), want)


class Layer(torch.autograd.Function):
    """How a model uses the layer in training."""

    @staticmethod
    def forward(ctx, x, w, w_t, a, b):
        ctx.kept, ctx.w_t = training.checkpoint(x, fine=True), w_t
        ctx.save_for_backward(a, b)
        return rtl.sparse_linear(x, w, a, b, 0.5)

    @staticmethod
    def backward(ctx, g):
        dx, da, db = training.sparse_linear_backward(g.contiguous(), ctx.kept, ctx.w_t, *ctx.saved_tensors, 0.5)
        return dx, None, None, da, db


def test_inside_an_autograd_function():
    x, w, a, b = rand(2, 20, 64).requires_grad_(), rand(32, 64), rand(4, 64).requires_grad_(), rand(32, 4).requires_grad_()
    w_t, g = w.t().contiguous(), rand(2, 20, 32)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        y = Layer.apply(x, w, w_t, a, b)
        y.backward(g)
    with torch.no_grad():
        want = training.sparse_linear_backward(g, training.checkpoint(x, fine=True), w_t, a, b, 0.5)
        assert torch.equal(y, rtl.sparse_linear(x, w, a, b, 0.5))
    for t, grad in zip((x, a, b), want):
        assert torch.equal(t.grad, grad)
