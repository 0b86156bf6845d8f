"""What w4.Weight takes: the kernels read numel() bytes from the data pointer on."""
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import w4  # noqa: E402


def test_other_types_and_host_bytes_are_refused():
    need = w4.packed_bytes(16, 128, 128)
    for dtype in (torch.float32, torch.int8, torch.bool):
        with pytest.raises(TypeError):
            w4.Weight(torch.zeros(need, dtype=dtype), 16, 128, 128, False)
    with pytest.raises(ValueError):
        w4.Weight(torch.zeros(need, dtype=torch.uint8), 16, 128, 128, False)


@pytest.mark.gpu
def test_bytes_that_do_not_lie_side_by_side_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    need = w4.packed_bytes(16, 128, 128)
    one = torch.zeros(1, dtype=torch.uint8, device="cuda:0")
    for packed in (one.expand(need), torch.zeros(2 * need, dtype=torch.uint8, device="cuda:0")[::2]):
        with pytest.raises(ValueError):
            w4.Weight(packed, 16, 128, 128, False)
    whole = torch.zeros(need, dtype=torch.uint8, device="cuda:0")
    x = torch.ones(1, 128, dtype=torch.bfloat16, device="cuda:0")
    assert (w4.linear(x, w4.Weight(whole, 16, 128, 128, False)) == 0).all()
