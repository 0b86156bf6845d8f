"""The attention kernels' barriers release LDS tiles to the next direct copies: every one is passed only with the
wavefront's own copies arrived and its LDS reads returned, in the built code and not by the compiler's order alone."""
import os
import re
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import listing  # noqa: E402

from activation_sparse_gemm_token_amd import library_path  # noqa: E402

if not os.path.exists(library_path) or not os.path.exists(os.path.join(listing.LLVM, "llvm-objdump")):
    pytest.skip("needs the built library and its toolchain", allow_module_level=True)


def test_barriers_wait_for_copies_and_reads(tmp_path):
    kernels = {}
    for path in listing.code_objects(library_path, str(tmp_path)):
        kernels.update(listing.instructions(path, "attn_(forward|dq|dkv)_kernel"))
    assert len(kernels) == 8 + 4 + 4                               # two types, four widths
    for name, lines in kernels.items():
        at = [i for i, line in enumerate(lines) if line.startswith("s_barrier")]
        assert at, name
        for i in at:
            wait = re.match(r"s_waitcnt (.*)", lines[i - 1])
            assert wait and {"vmcnt(0)", "lgkmcnt(0)"} <= set(wait[1].split()), (name, i, lines[i - 3:i + 1])
