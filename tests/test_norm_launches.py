"""Layer norm's launches at the largest sizes that its header allows, recorded on the host."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import launches  # noqa: E402

P = 1 << 20
HIDDEN = "u32(0)", "vp(None)"                                      # flags, stream


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return launches.recorder(str(tmp_path_factory.mktemp("recorder")))


def forward(rows, c):
    return "rtl_layer_norm", [P, 1, rows, c, 0, c, 0, 0, 0, 0, "f32(0)", "f32(1e-5)", P, 0, c, 0, 0, *HIDDEN]


def backward(rows, c, batch=1, groups=1):
    """Rows one after another: of one sequence, or one of each."""
    b, t = (0, rows) if batch == 1 else (c, 1)
    return "rtl_layer_norm_backward", [P, b, c, P, b, c, P, P, batch, t, c, P, c, "f32(0)", groups, P, b, c, P, P, P, 1 << 50, *HIDDEN]


CHANNELS = [1, 16, 128, 256, 512, 1024, 2048, 4096, 8192, 8193, 16384, 16385, 32768]


@pytest.mark.parametrize("rows", [1, (1 << 21) + 1, 1 << 22, (1 << 30) - 1])
def test_every_row_of_a_large_tensor(lib, rows):
    """Each launch keeps within a grid's limits, and the forward pass has threads for every row (16 to 1024 a row)."""
    calls = [forward(rows, c) for c in CHANNELS]
    for c, (status, got) in zip(CHANNELS, launches.record(lib, calls)):
        assert status == 0 and len(got) == 1
        (grid, block), per_row = got[0], 16 if c <= 128 else 32 if c <= 256 else 64 if c <= 2048 else 256 if c <= 8192 else 1024
        assert launches.launchable(grid, block), (c, grid, block)
        assert grid[0] * grid[1] * grid[2] * (block[0] // per_row) >= rows, (c, grid, block)


def test_gradients_of_many_rows_and_sequences(lib):
    calls = [backward(n, c) for c in CHANNELS for n in (1, 1 << 22, (1 << 30) - 1)]
    calls += [backward(n, c, n, n) for c in CHANNELS for n in (70_000, 1 << 22, (1 << 30) - 1)]
    for call, (status, got) in zip(calls, launches.record(lib, calls)):
        assert status == 0 and got
        assert all(launches.launchable(*g) for g in got), (call, got)


def test_up_to_two_to_the_31_rows(lib):
    """batch * tokens < 2^31: the last number below it, and the first that is not."""
    most = (1 << 31) - 1
    for c in (1, 9000):
        for (status, got), fits in zip(launches.record(lib, [forward(most, c), backward(most, c), forward((1 << 30) + 1, c),
                                                            backward(most, c, most, most), forward(most + 1, c)]), (1, 1, 1, 1, 0)):
            assert status == (0 if fits else 2)                    # RTL_ERR_BAD_SHAPE
            assert bool(got) == bool(fits) and all(launches.launchable(*g) for g in got)
