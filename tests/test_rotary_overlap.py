"""Which outputs rotary.rope takes: the overlap check, on CPU tensors."""
import itertools
import random

import pytest

torch = pytest.importorskip("torch")

from activation_sparse_gemm_token_amd import rotary  # noqa: E402


def _elements(t):
    at = [t.data_ptr()]
    for n, s in zip(t.shape, t.stride()):
        at = [p + i * s * t.element_size() for p in at for i in range(n)]
    return set(at)


def _slices():
    """Query, key and value slices of one projection's output, every order of its dimensions in memory."""
    for b, t, hq, hk, d in ((2, 5, 6, 2, 4), (3, 1, 1, 1, 2), (1, 4, 3, 3, 8), (2, 3, 1, 4, 1)):
        heads = hq + 2 * hk
        for order in itertools.permutations(range(3)):
            shape = [(b, t, heads)[i] for i in order]
            back = [order.index(i) for i in range(3)]
            x = torch.empty(*shape, d).permute(*back, 3)
            yield x[:, :, :hq], x[:, :, hq:hq + hk], x[:, :, hq + hk:]
    x = torch.empty(2, 5, 4, 3, 8)                                 # q, k and v beside each other in every head
    yield x[:, :, :, 0], x[:, :, :, 1], x[:, :, :, 2]


def test_slices_of_one_tensor_are_apart():
    for parts in _slices():
        for a, b in itertools.permutations(parts, 2):
            assert rotary._apart(a, b), (a.shape, a.stride(), b.shape)
            for t in (a[0], a[:, :1], a[:1]):
                assert rotary._apart(t, b[0] if t.dim() == 3 else b[:, :t.shape[1]][:t.shape[0]])


def test_in_place_calls_on_slices_pass_the_check():
    for q, k, v in _slices():
        rotary._check_overlap((("x", q, q), ("k", k, k)), [q, k])
        rotary._check_overlap((("x", q, None), ("k", k, v)), [torch.empty_like(q), v])
        with pytest.raises(ValueError):
            rotary._check_overlap((("x", q, k), ("k", k, None)), [k, torch.empty_like(k)])


def test_never_apart_when_an_element_is_shared():
    """Random views of one buffer: apart is only said of views that are, and said
    of all that are slices along one dimension."""
    rng = random.Random(4)
    buf = torch.empty(4000)
    shared = 0
    for _ in range(4000):
        dims = rng.choice([3, 4])
        shape = [rng.randint(1, 4) for _ in range(dims - 1)] + [rng.choice([1, 2, 4])]
        stride = [rng.choice([0, 1, 2, 3, 4, 6, 8, 12, 24, 32, 48, 96]) for _ in range(dims - 1)] + [1]
        other = list(shape)
        other[-2] = rng.randint(1, 4)
        a = buf.as_strided(shape, stride, rng.randint(0, 40))
        b = buf.as_strided(other, stride if rng.random() < 0.9 else stride[::-1], rng.randint(0, 120))
        meet = bool(_elements(a) & _elements(b))
        shared += meet
        if meet:
            assert not rotary._apart(a, b) and not rotary._apart(b, a)
        elif a.stride() == b.stride():
            assert rotary._apart(a, b) and rotary._apart(b, a)
    assert 500 < shared < 3500


def test_other_strides_are_not_called_apart():
    c = torch.empty(8, 8, 4)
    assert not rotary._apart(c[:4, :4], c.transpose(0, 1)[:4, :4])
