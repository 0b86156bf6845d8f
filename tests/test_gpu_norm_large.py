"""Layer norm of tensors at the far end of what its header allows, in place; memory is given back."""
import gc

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import norm  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def give_back():
    gc.collect()
    torch.cuda.empty_cache()
    yield
    gc.collect()
    torch.cuda.empty_cache()


def in_place(rows, c, seed):
    """Zeros with some rows that are not, at both ends and on both sides of 2^21 and 2^22: as those rows by themselves."""
    at = sorted({i for i in (0, 1, (1 << 21) - 1, 1 << 21, (1 << 22) - 1, 1 << 22, (1 << 30) - 1, 1 << 30, rows - 2, rows - 1) if i < rows})
    some = torch.randn(len(at), c, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)
    x = torch.zeros(rows, c, dtype=BF, device=DEV)
    x[at] = some
    assert norm.layer_norm(x, out=x).data_ptr() == x.data_ptr()
    assert torch.equal(x[at], norm.layer_norm(some))
    x[at] = 0
    assert all(not part.any() for part in x.split(1 << 24))


def test_more_workgroups_of_1024_than_a_dimension_holds():
    in_place((1 << 22) + 1, 8200, 1)                               # 69 GB


def test_more_than_two_to_the_30_rows():
    in_place((1 << 30) + 9, 8, 2)
