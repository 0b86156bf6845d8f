"""Outputs of the operators beside the layer that overlap what they are formed from."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import training, w4  # noqa: E402

DEV = "cuda:0"


def test_linear_into_its_input_is_refused():
    """Other workgroups still read x while the first write y."""
    n = k = 256
    codes = torch.randint(0, 256, (n, k // 2), device=DEV, dtype=torch.uint8)
    weight = w4.pack(codes, torch.ones(n, k // 128, device=DEV, dtype=torch.bfloat16))
    rows = torch.randn(6, k, device=DEV).bfloat16()
    x, before = rows[:4], rows.clone()
    for out in (x, rows[2:6], x.view(2, 2, k)):
        with pytest.raises(ValueError):
            w4.linear(x.view(*out.shape[:-1], k), weight, out=out)
    assert torch.equal(rows, before)
    y = w4.linear(rows[:3], weight, out=rows[3:])                  # side by side is fine
    assert torch.equal(y, w4.linear(before[:3], weight)) and torch.equal(rows[:3], before[:3])
    with pytest.raises(ValueError):
        w4.linear(x, weight, out=weight.packed[:2 * 4 * n].view(torch.bfloat16).view(4, n))


def test_unpack_into_its_codes_is_refused():
    kept = training.checkpoint(torch.randn(4, 64, device=DEV).bfloat16())
    room = torch.empty(4 * 64 * 2, dtype=torch.uint8, device=DEV)
    codes = room[:4 * 64].view(torch.int8).view(4, 64)
    codes.copy_(kept.codes)
    with pytest.raises(ValueError):
        training.unpack(codes, kept.exps, out=room.view(torch.bfloat16).view(4, 64))
    assert torch.equal(training.unpack(codes, kept.exps), kept.unpack())
