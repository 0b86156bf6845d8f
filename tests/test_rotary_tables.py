"""Arguments of the frequency tables that have no table."""
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import rotary  # noqa: E402


@pytest.mark.parametrize("bad", [dict(base=1.0), dict(base=0.5), dict(base=0.0), dict(base=-2.0), dict(base=float("nan")),
                                 dict(factor=float("nan")), dict(factor=0.5), dict(fast_turns=1.0), dict(slow_turns=0.0)])
def test_by_parts_refuses_what_has_no_turns(bad):
    """With a base of 1 every pair turns alike, so no pair turns ``fast_turns`` times."""
    with pytest.raises(ValueError):
        rotary.frequencies_by_parts(64, **{"factor": 4.0, "trained_length": 4096, **bad})
