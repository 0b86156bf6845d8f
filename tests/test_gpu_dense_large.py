"""Dense linears of tensors a few bytes below 2 GiB: their last rows, whose offsets are the largest."""
import gc

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import dense  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def give_back():
    gc.collect()
    torch.cuda.empty_cache()
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,k,back", [((2 ** 31 - 1) // 48, 24, 24, True), (1 << 26, 9, 8, False)])
def test_last_rows(m, n, k, back):
    """Sums of at most 24 products of eighths, exact in fp32: a result is half a step of bf16 off at most."""
    g = torch.Generator(device=DEV).manual_seed(m)
    eighths = lambda *s: (torch.randint(-8, 9, s, generator=g, device=DEV, dtype=torch.int8).to(BF) / 8)  # noqa: E731
    x, w = eighths(m, k), eighths(n, k)
    y = dense.linear(x, w)
    dy = eighths(m, n) if back else None
    dx = dense.linear_backward(dy, x, w, need_dw=False, need_dbias=False)[0] if back else None
    for part in (slice(0, 300), slice(m // 2, m // 2 + 300), slice(m - 300, m)):
        want = x[part].double() @ w.double().t()
        assert ((y[part].double() - want).abs() <= 2.0 ** -8 * want.abs()).all()
        if back:
            want = dy[part].double() @ w.double()
            assert ((dx[part].double() - want).abs() <= 2.0 ** -8 * want.abs()).all()
