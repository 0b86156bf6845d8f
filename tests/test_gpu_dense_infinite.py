"""Dense linears whose sums are infinite, in fp32 or in the type that z is kept in: activations and slopes take
their limits there, and a sum that is not a number stays one."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import dense  # noqa: E402

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16
ACTS = ["gelu", "gelu_tanh", "silu"]


def diagonal(values, dtype, n):
    """x [len(values), 8] and w [n, 8] with x w^T = values in column 0 and 1 elsewhere: the value is a product of two
    that the type holds."""
    x = torch.zeros(len(values), 8, dtype=dtype, device=DEV)
    x[:, 1] = 1
    w = torch.zeros(n, 8, dtype=dtype, device=DEV)
    w[:, 1] = 1
    w[0, 0], w[0, 1] = 256, 0
    x[:, 0] = torch.tensor([v / 256 for v in values], dtype=torch.float64).to(dtype)
    return x, w


@pytest.mark.parametrize("rows", [4, 60])
@pytest.mark.parametrize("act", ACTS)
def test_z_past_fp16(act, rows):
    """Finite tensors whose z is finite in fp32 and infinite in fp16, in the kernel for few rows and in tiles."""
    values = [70144.0, -70144.0, 2.0, -2.0] * (rows // 4)
    x, w = diagonal(values, HF, 16)
    y, z = dense.linear(x, w, activation=act, keep=True)
    assert torch.isposinf(z[0::4, 0]).all() and torch.isneginf(z[1::4, 0]).all()
    assert torch.isposinf(y[0::4, 0]).all() and (y[1::4, 0] == 0).all()
    dy = torch.ones_like(y)
    dx, dw, db, _ = dense.linear_backward(dy, x, w, z, activation=act)
    assert all(torch.isfinite(t).all() for t in (dx, dw, db))
    # Column 0 alone: dz is the slope, 1 above and 0 below.
    dy[:, 1:] = 0
    dx, dw, db, _ = dense.linear_backward(dy, x, w, z, activation=act)
    assert (dx[0::4, 0] == 256).all() and (dx[1::4, 0] == 0).all()
    # s(2) + s(-2) = 1 for every slope here, so each four rows add 2 up; two slopes rounded to fp16 (2^-11 each).
    assert abs(float(db[0]) - rows / 2) <= rows / 2 * 2.0 ** -9


@pytest.mark.parametrize("z_type", [BF, torch.float32])
@pytest.mark.parametrize("act", ACTS)
def test_an_infinite_sum(act, z_type):
    """Past fp32: the forward pass at both ends, then gradients (with a gate's) from an infinite z."""
    x, w = diagonal([0.0] * 4, BF, 16)
    x[0, 0], x[1, 0] = 3e38, -3e38
    y = dense.linear(x, w, activation=act)
    assert torch.isposinf(y[0, 0]) and y[1, 0] == 0 and torch.isfinite(y[2:]).all()
    z = torch.ones(4, 16, dtype=z_type, device=DEV)
    z[0, 0], z[1, 0], z[2, 0] = math.inf, -math.inf, math.nan
    x[:, 0] = 0
    dy, gate = torch.ones(4, 16, dtype=BF, device=DEV), torch.ones(16, dtype=BF, device=DEV)
    dy[0, 0] = 0                                                   # of +inf the activation is infinite: 0 * inf is not a number
    dx, dw, db, dg = dense.linear_backward(dy[:2], x[:2], w, z[:2], activation=act, gate=gate)
    assert all(torch.isfinite(t).all() for t in (dx, dw, db)) and dx[1, 0] == 0
    dg = dense.linear_backward(dy[1:2], x[1:2], w, z[1:2], activation=act, gate=gate)[3]
    assert torch.isfinite(dg).all() and dg[0] == 0
    dg = dense.linear_backward(torch.ones_like(dy[:1]), x[:1], w, z[:1], activation=act, gate=gate)[3]
    assert torch.isposinf(dg[0]) and torch.isfinite(dg[1:]).all()
    dx = dense.linear_backward(dy[2:3], x[2:3], w, z[2:3], activation=act)[0]
    assert torch.isnan(dx[0, 0])


@pytest.mark.parametrize("act", ACTS)
def test_a_sum_that_is_not_a_number(act):
    x, w = diagonal([math.nan, 1.0], BF, 16)
    y = dense.linear(x, w, activation=act)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1]).all()
