"""training.backward_form on the host: the forms that sizes take, and its refusals."""
import ctypes
import random

import pytest

pytest.importorskip("torch")

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import training  # noqa: E402


def test_refusals():
    for bad in ((-1, 64, 128, 16), (8, 62, 128, 16), (8, 64, 126, 16), (8, 64, 128, 129), (8, 64, 128, -1), (1 << 23, 64, 128, 0)):
        with pytest.raises(rtl.RtlError) as e:
            training.backward_form(*bad)
        assert e.value.status == 2
    assert training._fn("rtl_sparse_linear_backward_form")(8, 64, 128, 16, ctypes.POINTER(ctypes.c_int64)()) == 1


def test_ranges_cover_their_length():
    """No range is empty, and rows are long enough for 16-byte copies where they are copied so."""
    rng = random.Random(2)
    for _ in range(500):
        m, n, k = int(2 ** rng.uniform(0, 13)), 4 * int(2 ** rng.uniform(0, 11)), 4 * int(2 ** rng.uniform(0, 11))
        columns, ranges, length, over_n, over_k, tokens = training.backward_form(m, n, k, rng.choice([0, 4, 33, 128]))
        steps = -(-n // 64)
        per = -(-steps // ranges)
        assert columns in (64, 192, 256) and 1 <= ranges <= 16 and (ranges - 1) * per < steps
        assert length == n if columns == 64 or n % 8 == 0 else length == n + 4
        assert over_n % 256 == over_k % 256 == tokens % 128 == 0 and min(over_n, over_k, tokens) > 0
