"""w4.linear past 64 rows, on both sides of where tiles of 64 rows take over."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import w4  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("m,k,n", [(64, 1408, 4099), (100, 1408, 8000), (129, 1408, 8100), (250, 1408, 4099), (1000, 1152, 1030),
                                   (1025, 1152, 900), (4097, 1280, 260), (70, 1280, 9000)])
def test_many_rows(m, k, n, group, zeros):
    """Against fp64.  Products are exact, the sums fp32: a product with 1 + q / 16 and
    its share of the sum of x each pass at most k / 32 + 20 roundings of magnitudes
    below 2 (1 + q / 16) < 4 times |x|, times 16 s; then the result's own half step."""
    print("[w4]", m, k, n, group, zeros, file=sys.stderr, flush=True)
    g = torch.Generator(device=DEV).manual_seed(m + n)
    x = torch.randn(m, k, generator=g, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = (0.005 * torch.rand(n, k // group, generator=g, device=DEV) + 0.002).bfloat16()
    z = torch.randint(0, 16, (n, k // group), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    y = w4.linear(x, w4.pack(codes, scales, z, group=group))
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(1).double().view(n, -1, group)
    w = ((q - (8.0 if z is None else z.double()[..., None])) * scales.double()[..., None]).view(n, k)
    want = x.double() @ w.t().contiguous()
    size = x.double().abs() @ (16 * scales.double()).repeat_interleave(group, 1).t().contiguous()
    tol = 2.0 ** -8 * want.abs() + (k / 32 + 20) * 2.0 ** -24 * 4 * size
    assert int(((y.double() - want).abs() > tol).sum()) == 0
    assert torch.equal(y[-7:], w4.linear(x, w4.pack(codes, scales, z, group=group))[-7:])
