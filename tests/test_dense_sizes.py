"""The dense linear's sizes on the host: every tensor below 2 GiB, to the byte."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import launches  # noqa: E402

P = 1 << 20
OK, SHAPE = 0, 2
LIMIT = 1 << 31


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return launches.recorder(str(tmp_path_factory.mktemp("recorder")))


def forward(m, n, k):
    return "rtl_linear", [P, P, 0, 0, 1, 0, 0, m, n, k, P, 0, P, 1 << 50, "u32(0)", "vp(None)"]


def backward(m, n, k):
    return "rtl_linear_backward", [P, P, P, 0, 0, 1, 0, m, n, k, P, P, P, 0, P, 1 << 50, "u32(0)", "vp(None)"]


# (M, N, K), and whether the backward pass's rows of dz, N rounded up to 8, stay below 2 GiB as well.
FITS = [((LIMIT - 1) // 48, 24, 24, True), ((LIMIT - 1) // 80, 40, 40, True), (24, (LIMIT - 1) // 80, 40, True), (7, 32, (1 << 25) - 8, True),
        (1 << 26, 9, 8, False), ((LIMIT - 1) // 18, 9, 8, False), (3, (1 << 25) - 1, 8, True)]
PAST = [((LIMIT - 1) // 48 + 1, 24, 24), (24, (LIMIT - 1) // 80 + 1, 40), ((LIMIT - 1) // 18 + 1, 9, 8), (1 << 27, 8, 8)]


def test_the_largest_tensors(lib):
    for (m, n, k, both), (status, got) in zip(FITS, launches.record(lib, [forward(*f[:3]) for f in FITS])):
        assert max(m * k, n * k, m * n) * 2 < LIMIT and status == OK and got and all(launches.launchable(*g) for g in got), (m, n, k)
    for (m, n, k, both), (status, got) in zip(FITS, launches.record(lib, [backward(*f[:3]) for f in FITS])):
        assert status == (OK if both else SHAPE) and all(launches.launchable(*g) for g in got), (m, n, k)


def test_the_first_past_them(lib):
    calls = [call(*p) for p in PAST for call in (forward, backward)]
    assert all(max(m * k, n * k, m * n) * 2 >= LIMIT for m, n, k in PAST)
    assert all(status == SHAPE and not got for status, got in launches.record(lib, calls))
