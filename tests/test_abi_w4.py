"""The 4-bit linear's entry points on the host, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import w4  # noqa: E402

OK, NULLP, SHAPE, MISAL, WS, NODEV, ARCH, HIP, FLAGS = range(9)
P, P2, P3, P4 = 0x10000, 0x20000, 0x30000, 0x40000
BIG = 1 << 40


def _no_gpu():
    return torch.cuda.device_count() == 0


def _pack(c=P, s=P2, z=P3, n=20, k=256, group=64, flags=1, p=P4, size=BIG):
    return w4._fn("rtl_w4_pack")(c, s, z, n, k, group, flags, p, size, None)


def _linear(x=P, p=P2, size=BIG, m=3, n=20, k=256, group=64, flags=1, y=P3):
    return w4._fn("rtl_w4_linear")(x, p, size, m, n, k, group, flags, y, None)


def test_packed_bytes():
    for n, k, group, zeros in [(16, 128, 128, False), (17, 128, 128, True), (4099, 12288, 64, True), (1, 32, 32, False)]:
        tiles = -(-n // 16) * -(-k // 128)
        assert w4.packed_bytes(n, k, group, zeros) == tiles * (1024 + 16 * (128 // group) * (4 if zeros else 2))
    for bad in [(0, 128, 32), (16, 0, 32), (16, 100, 32), (16, 128, 16), (16, 128, 256), (-1, 128, 32), (1 << 31, 128, 32)]:
        assert w4.packed_bytes(*bad) == 0
    assert w4._fn("rtl_w4_packed_bytes")(16, 128, 32, 2) == 0
    assert w4.packed_bytes(1 << 20, 1 << 20, 128) == (1 << 16) * (1 << 13) * (1024 + 32)


@pytest.mark.parametrize("call", [_pack, _linear])
def test_refusals(call):
    for bad in (dict(n=0), dict(n=-1), dict(k=0), dict(k=100), dict(group=16), dict(group=0), dict(n=1 << 31),
                dict(k=(1 << 22) + 128)):
        assert call(**bad) == SHAPE, bad
    assert call(flags=2) == FLAGS
    assert call(p=None) == NULLP and call(p=P2 + 8) == MISAL
    need = w4.packed_bytes(20, 256, 64, True)
    assert call(size=need - 1) == WS
    if _no_gpu():
        assert call(size=need) == NODEV


def test_pack_and_linear_arguments():
    for bad in (dict(c=None), dict(s=None), dict(z=None)):
        assert _pack(**bad) == NULLP
    for bad in (dict(c=P + 4), dict(s=P2 + 2), dict(z=P3 + 1)):
        assert _pack(**bad) == MISAL
    assert _linear(x=None) == NULLP and _linear(y=None) == NULLP
    assert _linear(x=P + 8) == MISAL and _linear(y=P3 + 2) == MISAL
    assert _linear(m=-1) == SHAPE and _linear(m=w4.MAX_ROWS + 1) == SHAPE
    assert _linear(m=0, x=None, p=None, size=0, y=None) == OK
    if _no_gpu():
        assert _pack(z=None, flags=0) == NODEV and _linear(m=w4.MAX_ROWS) == NODEV


def test_binding_refusals():
    codes, scales = torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4.pack(codes, scales)                       # host tensors
    with pytest.raises(ValueError):
        w4.pack(codes, scales, group=48)
    with pytest.raises(ValueError):
        w4.pack(codes[:, :40], scales, group=128)
    with pytest.raises(TypeError):
        w4.pack(codes.int(), scales)
