"""Rotary positions on the GPU against a plain rotation in fp64.

Tolerance per element: half a step of the result's type, plus what fp32 loses
before that rounding.  Sine and cosine are off by at most 4 units of 2^-24
(the reduced angle rounded to fp32 moves them by less than one, the function
itself by two, the product with the scale by one), each of the two products
and their sum by one more of the magnitudes involved: 7 units of
2^-24 * scale * (|x0| + |x1|), taken as 8.  fp16 results below 2^-14 are
rounded to multiples of 2^-24: half of that is added."""
import itertools
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import rotary  # noqa: E402

DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def say(*a):
    print("[rotary]", *a, file=sys.stderr, flush=True)


def plain(x, pos, freq, layout, sections, scale, inverse):
    """fp64 on the host; also returns the magnitude |x0| + |x1| per element."""
    v = x.detach().cpu().double().numpy()
    f = freq.cpu().numpy()
    p = pos.cpu().numpy().astype(np.float64)
    half = f.shape[0]
    if sections is None:
        ang = p[..., None] * f
    else:
        ang = p[..., np.repeat(np.arange(len(sections)), sections)] * f if half else np.zeros(p.shape[:-1] + (0,))
    ang = np.broadcast_to(ang, v.shape[:-2] + (half,))
    c, s = scale * np.cos(ang)[..., None, :], scale * np.sin(ang)[..., None, :] * (-1 if inverse else 1)
    i0 = np.arange(half) if layout == "half" else 2 * np.arange(half)
    i1 = i0 + half if layout == "half" else i0 + 1
    y, mag = v.copy(), np.zeros_like(v)
    y[..., i0] = v[..., i0] * c - v[..., i1] * s
    y[..., i1] = v[..., i1] * c + v[..., i0] * s
    mag[..., i0] = mag[..., i1] = scale * (np.abs(v[..., i0]) + np.abs(v[..., i1]))
    return y, mag


def check(got, x, pos, freq, layout="half", sections=None, scale=1.0, inverse=False):
    ref, mag = plain(x, pos, freq, layout, sections, scale, inverse)
    out = got.detach().cpu().double().numpy()
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(ref) + 8 * 2.0 ** -24 * mag
    if x.dtype == torch.float16:
        tol = tol + (mag > 0) * 2.0 ** -25
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.abs(out - ref).max()}"


def make(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def freq(rot, **kw):
    return rotary.frequencies(rot, **kw).to(DEV)


@pytest.mark.parametrize("layout", rotary.LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("d,rot", [(128, 128), (96, 40), (64, 64), (80, 20), (33, 10), (5, 4), (2, 2), (1024, 1024),
                                   (256, 6), (64, 0), (1, 0)])
def test_layouts_types_and_partial_heads(layout, dtype, d, rot):
    say(layout, dtype, d, rot)
    x, k = make((2, 37, 6, d), dtype, 1), make((2, 37, 2, d), dtype, 2)
    pos = torch.arange(2 * 37, device=DEV).view(2, 37) * 3 - 11
    f = freq(rot)
    for inverse in (False, True):
        fn = rotary.rope_backward if inverse else rotary.rope
        y, ky = fn(x, pos, f, k=k, layout=layout, scale=1.25)
        check(y, x, pos, f, layout, None, 1.25, inverse)
        check(ky, k, pos, f, layout, None, 1.25, inverse)
        if rot < d:
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 40), (2, 3), (17, 1), (300, 5), (1153, 24), (0, 4), (5, 0)])
@pytest.mark.parametrize("layout", rotary.LAYOUTS)
def test_lengths(tokens, heads, layout):
    say(tokens, heads, layout)
    x = make((tokens, heads, 128), torch.bfloat16, tokens + heads)
    pos = torch.randint(0, 5000, (tokens,), generator=torch.Generator().manual_seed(3)).to(DEV)
    f = freq(128)
    y = rotary.rope(x, pos, f, layout=layout)
    assert y.shape == x.shape
    if x.numel():
        check(y, x, pos, f, layout)


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 27, -(2 ** 27)])
def test_far_positions(far):
    x = make((1, 64, 2, 64), torch.float32, 4)
    pos = (torch.arange(64, device=DEV) + far)[None]
    f = freq(64)
    check(rotary.rope(x, pos, f), x, pos, f)


@pytest.mark.parametrize("sections", [[8, 28, 28], [0, 32, 32], [64], [16, 16, 16, 16], [64, 0]])
def test_position_axes(sections):
    say(sections)
    x = make((2, 50, 3, 128), torch.bfloat16, 5)
    pos = torch.randint(0, 300, (2, 50, len(sections)), generator=torch.Generator().manual_seed(6)).to(DEV)
    f = freq(128)
    for layout in rotary.LAYOUTS:
        check(rotary.rope(x, pos, f, layout=layout, sections=sections), x, pos, f, layout, sections)
    shared = pos[0]
    check(rotary.rope(x, shared, f, sections=sections), x, shared[None].expand(2, -1, -1), f, "half", sections)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_strides_slices_and_broadcasts(dtype):
    f = freq(48)
    pos = torch.arange(33, device=DEV) * 7
    fused = make((3, 33, 10, 64), dtype, 7)                     # 6 query, 2 key, 2 value heads
    q, k = fused[:, :, :6], fused[:, :, 6:8]
    for layout in rotary.LAYOUTS:
        y, ky = rotary.rope(q, pos, f, k=k, layout=layout)
        check(y, q, pos[None].expand(3, -1), f, layout)
        check(ky, k, pos[None].expand(3, -1), f, layout)
        swapped = make((3, 4, 33, 64), dtype, 8).transpose(1, 2)  # heads before tokens
        check(rotary.rope(swapped, pos, f, layout=layout), swapped, pos[None].expand(3, -1), f, layout)
        odd = make((3 * 33 * 2 * 65 + 1,), dtype, 9)[1:].view(3, 33, 2, 65)[..., :64]   # no alignment beyond an element
        check(rotary.rope(odd, pos, f, layout=layout), odd, pos[None].expand(3, -1), f, layout)
        wide = make((3, 33, 1, 64), dtype, 10).expand(3, 33, 5, 64)   # one head read five times
        check(rotary.rope(wide, pos, f, layout=layout), wide, pos[None].expand(3, -1), f, layout)


def test_in_place_leaves_everything_else():
    f = freq(40)
    pos = torch.arange(70, device=DEV).view(2, 35)
    fused = make((2, 35, 9, 96), torch.bfloat16, 11)
    q, k = fused[:, :, :5], fused[:, :, 5:7]
    before = fused.clone()
    want, kwant = rotary.rope(q, pos, f, k=k)
    y, ky = rotary.rope(q, pos, f, k=k, out=q, k_out=k)
    assert y.data_ptr() == q.data_ptr() and ky.data_ptr() == k.data_ptr()
    assert torch.equal(q, want) and torch.equal(k, kwant)
    assert torch.equal(fused[:, :, 7:], before[:, :, 7:])


def test_backward_is_the_transpose_and_matches_differences():
    f = freq(24)
    pos = torch.arange(9, device=DEV) * 1000
    for layout in rotary.LAYOUTS:
        x, g = make((9, 2, 32), torch.float32, 12), make((9, 2, 32), torch.float32, 13)
        y, dx = rotary.rope(x, pos, f, layout=layout, scale=1.5), rotary.rope_backward(g, pos, f, layout=layout, scale=1.5)
        a, b = (y.double() * g.double()).sum().item(), (x.double() * dx.double()).sum().item()
        bound = 16 * 2.0 ** -24 * 1.5 * 2 * (x.double().abs().sum() * g.double().abs().max()).item()
        assert abs(a - b) <= bound
        # a linear map: any step of the difference gives the directional derivative
        e = make((9, 2, 32), torch.float32, 14)
        diff = ((rotary.rope(x + e, pos, f, layout=layout, scale=1.5).double() - y.double()) * g.double()).sum().item()
        want = (e.double() * dx.double()).sum().item()
        assert abs(diff - want) <= 3 * bound + 16 * 2.0 ** -24 * 3 * (e.double().abs().sum() * g.double().abs().max()).item()


def test_non_finite_values_stay_in_their_pair():
    x = make((4, 1, 8), torch.bfloat16, 15)
    x[1, 0, 1], x[2, 0, 0] = float("nan"), float("inf")
    y = rotary.rope(x, torch.arange(4, device=DEV), freq(8)).float()
    ok = torch.ones_like(y, dtype=torch.bool)
    ok[1, 0, [1, 5]] = False
    ok[2, 0, [0, 4]] = False
    assert torch.isfinite(y[ok]).all() and torch.isnan(y[1, 0, [1, 5]]).all() and not torch.isfinite(y[2, 0, 0])


def test_streams_graph_and_repeats():
    x, f = make((2, 65, 4, 128), torch.bfloat16, 16), freq(128)
    pos = torch.arange(130, device=DEV).view(2, 65)
    want = rotary.rope(x, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = rotary.rope(x, pos, f)
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rotary.rope(x, pos, f, out=out)
    for i in range(4):
        x.copy_(make((2, 65, 4, 128), torch.bfloat16, 20 + i))
        eager = rotary.rope(x, pos, f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_offsets_past_32_bits():
    """A slice whose elements lie more than 2^31 elements into its tensor's storage and apart."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB free")
    store = torch.empty(2, (1 << 31) + 4096, dtype=torch.bfloat16, device=DEV)
    x = store[:, -3 * 2 * 64:].view(2, 3, 2, 64)
    x.copy_(make((2, 3, 2, 64), torch.bfloat16, 17))
    pos, f = torch.arange(6, device=DEV).view(2, 3), freq(64)
    want = x.clone()
    check(rotary.rope(x, pos, f), want, pos, f)
    rotary.rope(x, pos, f, out=x)
    check(x, want, pos, f)


def test_outputs_that_overlap_are_refused():
    f, pos = freq(16), torch.arange(4, device=DEV)
    x, k = make((4, 3, 16), torch.bfloat16, 18), make((4, 3, 16), torch.bfloat16, 19)
    fused = make((4, 8, 16), torch.bfloat16, 21)
    for kw in (dict(k=k, out=k), dict(k=x, out=x, k_out=x), dict(k=k, out=torch.empty_like(x), k_out=x),
               dict(out=torch.empty(4, 1, 16, dtype=x.dtype, device=DEV).expand(4, 3, 16))):
        with pytest.raises(ValueError):
            rotary.rope(x, pos, f, **kw)
    with pytest.raises(ValueError):
        rotary.rope(fused[:, :4], pos, f, k=fused[:, 3:5], out=fused[:, :4], k_out=fused[:, 3:5])
    with pytest.raises(ValueError):
        rotary.rope(fused[:, :4], pos, f, out=fused[:, 2:6])
    with pytest.raises(ValueError):
        rotary.rope(x, pos.cpu(), f)
    with pytest.raises(TypeError):
        rotary.rope(x, pos.int(), f)
    with pytest.raises(TypeError):
        rotary.rope(x, pos, f.float())
    # next to each other is fine
    want = rotary.rope(fused[:, :4].clone(), pos, f)
    got = rotary.rope(fused[:, :4], pos, f, out=fused[:, 4:])
    assert torch.equal(got, want)


def test_seeded_sweep():
    rng = np.random.default_rng(22)
    for i in range(30):
        d = int(rng.integers(1, 300))
        rot = 2 * int(rng.integers(0, d // 2 + 1))
        b, t, h, hk = int(rng.integers(1, 4)), int(rng.integers(1, 200)), int(rng.integers(1, 20)), int(rng.integers(1, 6))
        dtype, layout = DTYPES[int(rng.integers(3))], rotary.LAYOUTS[int(rng.integers(2))]
        pad = int(rng.integers(0, 9))
        say("sweep", i, b, t, h, hk, d, rot, dtype, layout, pad)
        x = make((b, t, h, d + pad), dtype, 50 + i)[..., :d]
        k = make((b, t, hk + 2, d), dtype, 90 + i)[:, :, 1:1 + hk]
        pos = torch.randint(-1000, 100000, (b, t), generator=torch.Generator().manual_seed(i)).to(DEV)
        f = freq(rot, linear=2.0, ntk=3.0)
        inverse = bool(rng.integers(2))
        y, ky = (rotary.rope_backward if inverse else rotary.rope)(x, pos, f, k=k, layout=layout, scale=0.7)
        check(y, x, pos, f, layout, None, 0.7, inverse)
        check(ky, k, pos, f, layout, None, 0.7, inverse)
