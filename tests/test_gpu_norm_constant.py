"""Layer norm of rows that are one value throughout: their sums are exact in fp32 (1000 C is a multiple of 8 below 2^24
such), so the mean is that value and the result exactly the bias, whatever the number of channels."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import norm  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("c", [1, 3, 7, 100, 129, 200, 500, 1000, 1023, 1028, 1152, 2000, 4099, 5000, 8191, 9000, 20001, 32768])
def test_constant_rows(c, dtype):
    value = torch.tensor([1000.0, -1000.0, 2.5, 0.0, 0.75, -992.0, 40.0], dtype=dtype, device=DEV)
    x = value[:, None].expand(7, c).contiguous()
    y, mean, rstd = norm.layer_norm(x, return_stats=True)
    assert torch.equal(mean, value.float()) and (y == 0).all()
    assert ((rstd.double() - 1e-5 ** -0.5).abs() <= 4 * 2.0 ** -24 * 1e-5 ** -0.5).all()
    w, b = torch.full((c,), 3.0, dtype=dtype, device=DEV), torch.full((c,), 0.5, dtype=dtype, device=DEV)
    assert (norm.layer_norm(x, w, b) == 0.5).all()
