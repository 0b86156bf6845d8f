"""4-bit linears on the GPU against the definition in fp64.

Tolerance per element: half a bf16 step of the result, plus the fp32 sums.
With a = 16 s |x| (2 + q / 16 + z / 16) per channel (both parts of the
difference that the kernel takes), an element passes at most `group`
additions inside its group and K / group + 3 across groups and wavefronts, and
five more roundings on the way (two fused multiply-adds, the scale, the group
sum's own): (group + K / group + 8) 2^-24 sum a."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import w4  # noqa: E402

DEV = "cuda:0"


def say(*a):
    print("[w4]", *a, file=sys.stderr, flush=True)


def make(m, k, n, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * m + 11 * n + 13 * k + group)
    x = torch.randn(m, k, generator=g).bfloat16()
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand(n, k // group, generator=g) * 0.02 + 0.001).bfloat16()
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    return x, codes, scales, z


def plain(x, codes, scales, z, group):
    q = np.stack([codes.numpy() & 15, codes.numpy() >> 4], -1).reshape(codes.shape[0], -1).astype(np.float64)
    zz = np.repeat(np.full(scales.shape, 8.0) if z is None else z.numpy().astype(np.float64), group, 1)
    s = np.repeat(scales.double().numpy(), group, 1)
    v = x.double().numpy()
    ref = v @ ((q - zz) * s).T
    size = np.abs(v) @ (16 * s * (2 + q / 16 + zz / 16)).T
    k = v.shape[1]
    return ref, 2.0 ** -8 * np.abs(ref) + (group + k // group + 8) * 2.0 ** -24 * size


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def run(x, codes, scales, z, group, **kw):
    xd, cd, sd, zd = dev(x, codes, scales, z)
    return w4.linear(xd, w4.pack(cd, sd, zd, group=group), **kw)


def check(got, ref, tol):
    out = got.double().cpu().numpy()
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(out - ref))}"


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("m,k,n", [(1, 128, 16), (1, 256, 1), (2, 384, 15), (3, 640, 17), (15, 1152, 333), (16, 2048, 64),
                                   (17, 128, 48), (31, 1280, 65), (32, 896, 160), (33, 1024, 100), (64, 1408, 257),
                                   (65, 256, 130), (200, 512, 70), (1, 12288, 40), (8, 1152, 4100),
                                   (3, 1088 * 2, 4112), (9, 1280, 4097), (16, 1152, 8200), (17, 1152, 8208), (32, 640, 8209),
                                   (33, 1152, 8200), (100, 384, 8193), (16, 1024, 33), (7, 896, 4096)])
def test_sizes(m, k, n, group, zeros):
    say(m, k, n, group, zeros)
    t = make(m, k, n, group, zeros)
    check(run(*t, group), *plain(*t, group))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("m,k,n", [(1, 2176, 4096), (8, 2176, 33), (8, 2304, 4097), (5, 2048, 130), (9, 2304, 5000),
                                   (16, 2176, 8192), (13, 2304, 8200), (16, 2048, 4100), (12, 6400, 70)])
def test_many_channels(m, k, n, group):
    """Either side of the sizes at which the channels, or the weight rows, are shared out among the wavefronts."""
    say(m, k, n, group)
    t = make(m, k, n, group, True)
    check(run(*t, group), *plain(*t, group))


@pytest.mark.parametrize("group,k", [(32, 32), (32, 96), (32, 160), (32, 4128), (64, 64), (64, 192), (64, 1088)])
@pytest.mark.parametrize("m", [1, 20, 50])
def test_channels_that_end_inside_a_tile(group, k, m):
    say(m, k, group)
    t = make(m, k, 37, group, True)
    check(run(*t, group), *plain(*t, group))


def test_full_range_of_codes_and_zero_points():
    k, group = 256, 64
    q = (torch.arange(16)[:, None] + torch.arange(k)[None]) % 16
    codes = (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8)
    x = (torch.eye(k) * 3).bfloat16()
    for z in [None] + [torch.full((16, k // group), v, dtype=torch.uint8) for v in (0, 7, 15)]:
        scales = torch.full((16, k // group), 0.5).bfloat16()
        got = run(x, codes, scales, z, group).float().cpu()
        want = 1.5 * (q - (8 if z is None else int(z[0, 0]))).T.float()
        assert torch.equal(got, want)            # small whole numbers times 1.5: nothing is rounded


def test_a_row_that_is_not_finite_stays_alone():
    t = make(20, 256, 40, 32, True)
    t[0][3, 5], t[0][18, 200] = float("nan"), float("inf")
    got = run(*t, 32)
    rows = [i for i in range(20) if i not in (3, 18)]
    clean = t[0].clone()
    clean[3], clean[18] = 0, 0
    ref, tol = plain(clean, *t[1:], 32)
    check(got[rows], ref[rows], tol[rows])
    assert not torch.isfinite(got[[3, 18]].float()).any()


def test_outliers_and_zero_rows():
    t = make(4, 1024, 64, 128, True)
    t[0][0] = 0
    t[0][1, ::100] *= 1000
    t[0][2] = t[0][2] * 2.0 ** 60
    t[0][3] = t[0][3] * 2.0 ** -60
    got = run(*t, 128)
    check(got, *plain(*t, 128))
    assert (got[0] == 0).all()


def test_memory_around_the_result_is_left_alone():
    for m, n in ((1, 17), (5, 99), (33, 70)):
        t = make(m, 256, n, 64, False)
        guard = torch.full((m * n + 512,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = guard[256:256 + m * n].view(m, n)
        run(*t, 64, out=out)
        assert (guard[:256] == 7).all() and (guard[256 + m * n:] == 7).all()
        check(out, *plain(*t, 64))


def test_pack_layout_is_the_documented_one():
    t = make(1, 160, 18, 32, True)
    cd, sd, zd = dev(*t[1:])
    got = w4.pack(cd, sd, zd, group=32)
    raw = got.packed.cpu().numpy()
    tiles = 2 * 2
    codes = raw[:tiles * 1024].view(np.uint32).reshape(2, 2, 64, 4)
    meta = raw[tiles * 1024:].view(np.uint32).reshape(2, 2, 16, 4)
    q = np.stack([t[1].numpy() & 15, t[1].numpy() >> 4], -1).reshape(18, 160)
    for nt in range(2):
        for kt in range(2):
            for lane in range(64):
                for j in range(4):
                    n, k = 16 * nt + lane % 16, 128 * kt + 32 * j + 8 * (lane // 16)
                    w = int(codes[nt, kt, lane, j])
                    for p in range(4):
                        for odd in range(2):
                            want = q[n, k + 2 * p + odd] if n < 18 and k < 160 else 0
                            assert w >> (4 * (p + 4 * odd)) & 15 == want
            for r in range(16):
                for g in range(4):
                    n, k = 16 * nt + r, 128 * kt + 32 * g
                    e = int(meta[nt, kt, r, g])
                    if n < 18 and k < 160:
                        assert e & 0xffff == int(t[2][n, k // 32].view(torch.int16)) & 0xffff
                        assert np.uint32(e & 0xffff0000).view(np.float32) == 1 + int(t[3][n, k // 32]) / 16
                    else:
                        assert e & 0xffff == 0


def test_batches_repeats_graph_and_streams():
    x, codes, scales, z = make(6, 512, 200, 128, True)
    xd, cd, sd, zd = dev(x, codes, scales, z)
    weight = w4.pack(cd, sd, zd)
    want = w4.linear(xd, weight)
    assert torch.equal(w4.linear(xd.view(2, 3, 512), weight).view(6, 200), want)
    # a row's result does not depend on the rows beside it in its 16
    assert torch.equal(w4.linear(xd[2:3].contiguous(), weight), want[2:3])
    assert w4.linear(xd[:0], weight).shape == (0, 200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = w4.linear(xd, weight)
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.linear(xd, weight, out=out)
    for i in range(4):
        xd.copy_(make(6, 512, 200, 128, True, seed=100 + i)[0])
        eager = w4.linear(xd, weight)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_refusals():
    x, codes, scales, z = dev(*make(2, 256, 32, 64, True))
    weight = w4.pack(codes, scales, z, group=64)
    with pytest.raises(ValueError):
        w4.linear(x[:, :192].contiguous(), weight)
    with pytest.raises(TypeError):
        w4.linear(x.float(), weight)
    with pytest.raises(ValueError):
        w4.linear(x, weight, out=torch.empty(2, 31, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        w4.pack(codes, scales[:, :3].contiguous(), z, group=64)
    with pytest.raises(TypeError):
        w4.pack(codes, scales.float(), z, group=64)
    with pytest.raises(rtl.RtlError) as e:
        w4.linear(x, w4.Weight(weight.packed[:-16], 32, 256, 64, True))
    assert e.value.status == 4


def test_seeded_sweep():
    rng = np.random.default_rng(3)
    for i in range(30):
        group = int(rng.choice(w4.GROUPS))
        m = int(2 ** rng.uniform(0, 8))
        k = group * int(rng.integers(1, max(2, 3000 // group)))
        n = int(2 ** rng.uniform(0, 13.3))
        zeros = bool(rng.integers(2))
        say("sweep", i, m, k, n, group, zeros)
        t = make(m, k, n, group, zeros, seed=i)
        check(run(*t, group), *plain(*t, group))


def test_many_rows_reread_the_weight():
    """More rows than one pass over the weight serves, and more tiles of rows
    than a chip has units."""
    t = make(3000, 256, 72, 64, True)
    check(run(*t, 64), *plain(*t, 64))
