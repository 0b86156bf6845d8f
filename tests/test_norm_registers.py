"""Layer norm's gradients: the forms whose comment says that a row and its sums fit their registers do."""
import os
import re
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import listing  # noqa: E402

from activation_sparse_gemm_token_amd import library_path  # noqa: E402

if not os.path.exists(library_path) or not os.path.exists(os.path.join(listing.LLVM, "llvm-readelf")):
    pytest.skip("needs the built library and its toolchain", allow_module_level=True)


def test_rows_that_fit_are_not_spilled(tmp_path):
    found = {}
    for name, (used, spills) in listing.registers(listing.code_objects(library_path, str(tmp_path))).items():
        m = re.search(r"norm_backward_kernelILi(\d)ELi(\d)ELi(\d+)ELi(\d+)E", name)
        if m:
            found[tuple(int(i) for i in m.groups())] = spills
    types, per_access, threads, elements = zip(*found)
    assert set(types) == {0, 1, 2} and set(per_access) == {1, 4, 8} and max(threads) == 1024 and set(elements) == {8, 16, 32}
    # Up to 8192 channels none; up to 16384 none by whole accesses of 16 bytes.
    bad = {k: v for k, v in found.items() if v and (k[2] < 1024 or (k[3] == 16 and k[1] == (4 if k[0] == 2 else 8)))}
    assert not bad, bad
