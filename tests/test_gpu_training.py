"""The 8-bit checkpoint and the layer's backward pass on the GPU against fp64
(tests/train_plain.py holds the definitions and the tolerances' derivation)."""
import sys

import numpy as np
import pytest

import oracle
from workloads import gen

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import training  # noqa: E402

sys.path.insert(0, __file__.rsplit("/", 1)[0])
import train_plain as plain  # noqa: E402

DEV = "cuda:0"


def say(*a):
    print("[training]", *a, file=sys.stderr, flush=True)


def to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def to_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def rand(shape, seed, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).bfloat16().to(DEV)


def inputs(m, k, law, seed):
    rng = np.random.default_rng(seed)
    if law == "mixture":
        return gen.mixture_bernoulli(rng, m, k)
    if law == "ties":
        return gen.tie_heavy(rng, m, k)
    if law == "gelu":
        return gen.gelu_of_normal(rng, m, k)
    bits = gen.uniform_bits(rng, (m, k), emax=100, span=220)       # 2^-120 .. 2^100, every block its own range
    bits[::3, :k // 2] = 0
    bits[1::5] &= 0x807f                                           # subnormal rows
    return bits


@pytest.mark.parametrize("law", ["mixture", "ties", "gelu", "wild"])
@pytest.mark.parametrize("m,k", [(1, 4), (1, 8), (3, 12), (5, 32), (2, 36), (7, 68), (4, 512), (33, 516), (9, 1024),
                                 (300, 1028), (130, 3072), (6, 12288), (9000, 64), (1, 12292)])
def test_checkpoint_is_the_defined_one(m, k, law):
    say(m, k, law)
    bits = inputs(m, k, law, m + k)
    x = to_dev(bits)
    kept = training.checkpoint(x)
    v = plain.bf16(x)
    codes, exps = plain.pack(v)
    assert np.array_equal(kept.codes.cpu().numpy(), codes)
    assert np.array_equal(kept.exps.cpu().numpy(), exps)
    _, idx, scale = rtl.sparsify_2of4(x)
    assert torch.equal(kept.idx, idx)
    mk = plain.mask(kept.idx.cpu().numpy(), k)
    lk = (mk * np.abs(v)).sum(1)
    got = kept.stats.cpu().double().numpy()
    if law != "wild":                                              # fp32 sums of positive numbers
        tol = (k / 128 + 16) * plain.U24
        assert (np.abs(got[:, 1] - lk) <= tol * lk).all()
        s = np.where(lk > 0, np.abs(v).sum(1) / np.where(lk > 0, lk, 1), 1)
        assert (np.abs(got[:, 0] - s) <= 3 * tol * s).all()
    stored = plain.values(codes, exps)
    y = kept.unpack()
    assert np.array_equal(plain.bf16(y), stored)                   # exact in bf16
    top = np.repeat(2.0 ** (exps.astype(float) - 133), 32, 1)[:, :k]
    assert (np.abs(stored - v) <= 0.5 * top).all()


def test_checkpoint_of_nothing_and_of_zeros():
    empty = training.checkpoint(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert empty.unpack().shape == (0, 64)
    kept = training.checkpoint(torch.zeros(3, 2, 40, dtype=torch.bfloat16, device=DEV))
    assert kept.unpack().shape == (3, 2, 40) and (kept.unpack() == 0).all() and (kept.exps == 0).all()
    assert (kept.stats[:, 0] == 1).all() and (kept.stats[:, 1] == 0).all()


def test_checkpoint_ignores_what_is_not_finite_elsewhere():
    """A row with an infinity or NaN leaves every other row as it was."""
    x = to_dev(inputs(8, 128, "mixture", 3))
    want = training.checkpoint(x)
    x[2, 17], x[5, 99] = float("inf"), float("nan")
    got = training.checkpoint(x)
    rows = [0, 1, 3, 4, 6, 7]
    for n in ("codes", "exps", "idx", "stats"):
        assert torch.equal(getattr(got, n)[rows], getattr(want, n)[rows])


def test_checkpoint_writes_only_its_rows():
    for m, k in ((3, 36), (5, 520), (2, 4)):
        x = rand((m, k), 4)
        guard = {}
        views = {}
        for name, dtype, width in (("codes", torch.int8, k), ("exps", torch.uint8, -(-k // 32)),
                                   ("idx", torch.uint8, -(-k // 8)), ("stats", torch.float32, 2)):
            buf = torch.full((m * width + 256,), 77, dtype=dtype, device=DEV)
            guard[name], views[name] = buf, buf[128:128 + m * width]
        st = training._fn("rtl_checkpoint_pack")(x.data_ptr(), m, k, *[views[n].data_ptr() for n in
                                                                      ("codes", "exps", "idx", "stats")], None)
        assert st == 0
        torch.cuda.synchronize()
        want = training.checkpoint(x)
        for name, buf in guard.items():
            n = views[name].numel()
            assert (buf[:128] == 77).all() and (buf[128 + n:] == 77).all(), name
            assert torch.equal(views[name], getattr(want, name).flatten()), name


def layer(m, n, k, r, seed=0, law="mixture"):
    x = to_dev(inputs(m, k, law, seed + m + k))
    return dict(kept=training.checkpoint(x), g=rand((m, n), seed + 1, 0.01), w_t=rand((k, n), seed + 2, 0.02),
                a=rand((r, k), seed + 3, 0.05) if r else None, b=rand((n, r), seed + 4, 0.05) if r else None)


def reference(t, alpha):
    kept = t["kept"]
    x = plain.values(kept.codes.cpu().numpy(), kept.exps.cpu().numpy())
    s, lk = kept.stats.cpu().double().numpy().T
    k, n = t["w_t"].shape
    a = plain.bf16(t["a"]) if t["a"] is not None else np.zeros((0, k))
    b = plain.bf16(t["b"]) if t["b"] is not None else np.zeros((n, 0))
    return plain.backward(plain.bf16(t["g"]), x, plain.mask(kept.idx.cpu().numpy(), k), s, lk, plain.bf16(t["w_t"]), a,
                          b, alpha)


def check(got, ref, tol):
    for name, y, want, t in zip(("dx", "da", "db"), got, ref, tol):
        if y is None:
            continue
        d = np.abs(plain.bf16(y).reshape(want.shape) - want)
        assert (d <= t).all(), f"{name}: {(~(d <= t)).sum()} of {d.size} off, worst {(d - t).max()}"


def run(t, alpha=1.0, **kw):
    return training.sparse_linear_backward(t["g"], t["kept"], t["w_t"], t["a"], t["b"], alpha, **kw)


SIZES = [(1, 4, 4, 1), (1, 8, 8, 4), (3, 12, 20, 5), (16, 64, 64, 16), (33, 100, 36, 32), (64, 128, 256, 33),
         (77, 264, 520, 16), (77, 260, 516, 64), (130, 520, 1028, 100), (257, 1024, 264, 128), (300, 132, 2052, 64),
         (700, 1000, 1000, 8), (1, 3000, 640, 128), (1100, 64, 96, 64)]


@pytest.mark.parametrize("m,n,k,r", SIZES)
def test_gradients(m, n, k, r):
    say(m, n, k, r)
    t = layer(m, n, k, r)
    check(run(t, 0.75), *reference(t, 0.75))


@pytest.mark.parametrize("m,n,k", [(1, 4, 4), (50, 260, 132), (300, 512, 512)])
def test_gradient_without_lora(m, n, k):
    t = layer(m, n, k, 0)
    got = run(t)
    assert got[1] is None and got[2] is None
    check(got, *reference(t, 1.0))


@pytest.mark.parametrize("law", ["ties", "gelu"])
def test_other_activations(law):
    t = layer(150, 264, 260, 24, law=law)
    check(run(t, -2.0), *reference(t, -2.0))


def test_only_what_is_asked_for():
    t = layer(90, 136, 260, 40)
    dx, da, db = run(t)
    only = run(t, need_lora=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    t["w_t"] = None
    lora = run(t, need_dx=False)
    assert lora[0] is None and torch.equal(lora[1], da) and torch.equal(lora[2], db)
    assert run(t, need_dx=False, need_lora=False) == (None, None, None)


def test_zero_rows_and_zero_gradients():
    x = to_dev(inputs(40, 128, "mixture", 9))
    x[7], x[31] = 0, 0
    t = layer(40, 64, 128, 16)
    t["kept"] = training.checkpoint(x)
    t["g"][3] = 0
    got = run(t)
    check(got, *reference(t, 1.0))
    assert (got[0][3] == 0).all() and torch.isfinite(got[0].float()).all()


def test_no_tokens():
    t = layer(4, 64, 128, 16)
    t["kept"] = training.checkpoint(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV))
    t["g"] = t["g"][:0]
    dx, da, db = run(t)
    assert dx.shape == (0, 128) and (da == 0).all() and (db == 0).all() and da.shape == (16, 128) and db.shape == (64, 16)


def test_against_differences():
    """Directional derivatives of the fp64 layer by central differences, at
    activations that the checkpoint holds exactly."""
    m, n, k, r, alpha = 20, 36, 64, 8, 0.5
    rng = np.random.default_rng(5)
    x = np.rint(rng.standard_normal((m, k)) * 20).clip(-63, 63) / 8
    x[:, ::32] = 8.0                                               # every block's largest: a step of 1/8
    t = dict(kept=training.checkpoint(torch.from_numpy(x).bfloat16().to(DEV)), g=rand((m, n), 1), w_t=rand((k, n), 2),
             a=rand((r, k), 3), b=rand((n, r), 4))
    assert np.array_equal(plain.bf16(t["kept"].unpack()), x)
    got = run(t, alpha)
    ref, tol = reference(t, alpha)
    check(got, ref, tol)
    g, w, a, b = plain.bf16(t["g"]), plain.bf16(t["w_t"]).T, plain.bf16(t["a"]), plain.bf16(t["b"])
    mk = plain.mask(t["kept"].idx.cpu().numpy(), k)

    def loss(x, a, b):
        return (g * plain.forward(x, mk, w, a, b, alpha)).sum()

    h = 1e-5
    for which, point in enumerate((x, a, b)):
        step = rng.standard_normal(point.shape)
        if which == 0:
            step = step * (x != 0)                                 # |x| has no derivative at 0
        args = [[x, a, b], [x, a, b]]
        args[0][which], args[1][which] = point + h * step, point - h * step
        diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        mine = (plain.bf16(got[which]) * step).sum()
        # fp64 differences: curvature h^2, cancellation 2^-52 |loss| / h
        slack = 1e-7 * (np.abs(ref[which]) * np.abs(step)).sum() + 2.0 ** -50 * (np.abs(g).sum() * 1e3) / h
        assert abs(mine - diff) <= (tol[which] * np.abs(step)).sum() + slack


def test_repeats_streams_and_shared_workspaces():
    t1, t2 = layer(200, 520, 516, 64), layer(90, 264, 1024, 32, seed=50)
    w1, w2 = run(t1), run(t2)
    for a, b in zip(w1, run(t1)):
        assert torch.equal(a, b)
    need = max(training.backward_workspace_bytes(200, 520, 516, 64), training.backward_workspace_bytes(90, 264, 1024, 32))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)       # NaN everywhere: nothing is read unwritten
    for a, b in zip(w1, run(t1, workspace=ws)):
        assert torch.equal(a, b)
    for a, b in zip(w2, run(t2, workspace=ws)):                          # a smaller layer after a larger one
        assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s1):
        o1 = run(t1)
    with torch.cuda.stream(s2):
        o2 = run(t2)
    torch.cuda.synchronize()
    for a, b in zip(w1 + w2, o1 + o2):
        assert torch.equal(a, b)


def test_captured_step():
    """Checkpoint and backward in one graph, replayed on new data."""
    m, n, k, r = 130, 264, 520, 16
    t = layer(m, n, k, r)
    x = to_dev(inputs(m, k, "mixture", 1))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = training.checkpoint(x)
        outs = training.sparse_linear_backward(t["g"], kept, t["w_t"], t["a"], t["b"])
    for i in range(4):
        x.copy_(to_dev(inputs(m, k, "mixture", 20 + i)))
        t["g"].copy_(rand((m, n), 60 + i, 0.01))
        eager = training.sparse_linear_backward(t["g"], training.checkpoint(x), t["w_t"], t["a"], t["b"])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)


def test_refusals():
    t = layer(8, 64, 128, 16)
    with pytest.raises(ValueError):
        training.sparse_linear_backward(t["g"][:4].contiguous(), t["kept"], t["w_t"], t["a"], t["b"])
    with pytest.raises(ValueError):
        training.sparse_linear_backward(t["g"], t["kept"], t["w_t"].t().contiguous(), t["a"], t["b"])
    with pytest.raises(ValueError):
        training.sparse_linear_backward(t["g"], t["kept"], None, t["a"], t["b"])
    with pytest.raises(ValueError):
        training.sparse_linear_backward(t["g"], t["kept"], t["w_t"], t["a"], None)
    with pytest.raises(rtl.RtlError) as e:
        run(t, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == 4
    odd = layer(8, 64, 128, 0)
    with pytest.raises(rtl.RtlError) as e:                              # N % 4
        training.sparse_linear_backward(rand((8, 62), 1), odd["kept"], rand((128, 62), 2))
    assert e.value.status == 2
    k = t["kept"]
    with pytest.raises(TypeError):
        training.Checkpoint(k.codes.view(torch.uint8), k.exps, k.idx, k.stats)
    with pytest.raises(ValueError):
        training.Checkpoint(k.codes, k.exps[:, :3].contiguous(), k.idx, k.stats)
    with pytest.raises(ValueError):
        training.Checkpoint(k.codes, k.exps, k.idx.cpu(), k.stats)


def test_forward_and_backward_meet():
    """The stored statistics are the forward's: y from the layer, and the fp64
    layer on the stored values with them, agree to the checkpoint's error."""
    m, n, k, r = 64, 128, 256, 16
    bits = inputs(m, k, "mixture", 2)
    x = to_dev(bits)
    kept = training.checkpoint(x)
    _, _, s_ref, _, _ = oracle.sparsify(bits)
    assert np.allclose(kept.stats[:, 0].cpu().numpy(), s_ref, rtol=1e-5, atol=0)


def test_seeded_sweep():
    rng = np.random.default_rng(8)
    for i in range(16):
        m, n, k = int(2 ** rng.uniform(0, 9.5)), 4 * int(2 ** rng.uniform(0, 8.5)), 4 * int(2 ** rng.uniform(0, 8.5))
        r, alpha = int(rng.integers(0, 129)), float(rng.uniform(-2, 2))
        say("sweep", i, m, n, k, r, alpha)
        t = layer(m, n, k, r, seed=100 * i, law=["mixture", "gelu", "ties"][i % 3])
        ws = torch.full((training.backward_workspace_bytes(m, n, k, r),), 0xff, dtype=torch.uint8, device=DEV)
        check(run(t, alpha, workspace=ws), *reference(t, alpha))


def test_a_gradient_row_that_is_not_finite_stays_alone():
    t = layer(70, 136, 260, 16)
    want = run(t)[0]
    t["g"][33, 5] = float("nan")
    dx = run(t)[0]
    rows = [i for i in range(70) if i != 33]
    assert torch.equal(dx[rows], want[rows]) and torch.isnan(dx[33].float()).all()


def test_large_tiles_and_ranges():
    """More than one round of tiles (256 columns), and a long contraction in
    many ranges; sampled rows against fp64."""
    for m, n, k, r in ((4100, 192, 4100, 16), (40, 12000, 200, 8), (1030, 320, 9000, 64)):
        say("large", m, n, k, r)
        t = layer(m, n, k, r)
        got = run(t, 0.5)
        rows = torch.tensor(sorted({0, 1, 255, 256, m // 2, m - 1} & set(range(m))), device=DEV)
        kept = t["kept"]
        part = dict(t, g=t["g"][rows], kept=training.Checkpoint(kept.codes[rows].contiguous(), kept.exps[rows].contiguous(),
                                                                kept.idx[rows].contiguous(), kept.stats[rows].contiguous()))
        ref, tol = reference(part, 0.5)
        d = np.abs(plain.bf16(got[0][rows]) - ref[0])
        assert (d <= tol[0]).all()
        # sums over all tokens: in fp64 on the device
        x = kept.unpack().double()
        mk = torch.from_numpy(plain.mask(kept.idx.cpu().numpy(), k)).to(DEV)
        s = kept.stats[:, :1].double()
        rest = x * (1 - s * mk)
        g, a, b = t["g"].double(), t["a"].double(), t["b"].double()
        u, tt = 0.5 * g @ b, 0.5 * rest @ a.t().contiguous()
        for got_i, want, size, lost in ((got[1], u.t().contiguous() @ rest, u.abs().t().contiguous() @ rest.abs(),
                                         plain.depth(n) * plain.U24 * (0.5 * g.abs() @ b.abs()).t().contiguous() @ rest.abs()),
                                        (got[2], g.t().contiguous() @ tt, g.abs().t().contiguous() @ tt.abs(),
                                         g.abs().t().contiguous() @ (plain.depth(k) * plain.U24 * 0.5 *
                                                                     (rest.abs() @ a.abs().t().contiguous())))):
            tol_i = plain.HALF_BF16 * want.abs() + (plain.depth(m) * plain.U24 + plain.U16 + 4 * plain.U24) * size + lost
            assert ((got_i.double() - want).abs() <= tol_i).all()


@pytest.mark.parametrize("m,n,k,r", [(1, 64, 64, 4), (15, 4, 4, 0), (16, 452, 60, 3), (63, 260, 516, 16), (64, 4096, 128, 0),
                                     (65, 4100, 68, 32), (130, 1000, 1004, 7), (200, 3000, 132, 64), (333, 516, 64, 128)])
def test_few_tokens(m, n, k, r):
    """Tiles of 64 tokens, one contraction range and several, tails in all three sizes."""
    say("few tokens", m, n, k, r)
    t = layer(m, n, k, r)
    ws = torch.full((training.backward_workspace_bytes(m, n, k, r),), 0xff, dtype=torch.uint8, device=DEV)
    got = run(t, -0.7, workspace=ws)
    check(got, *reference(t, -0.7))
    for a, b in zip(got, run(t, -0.7)):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("m,n,k", [(1944, 40, 1612), (640, 64, 6456), (66, 1032, 8248), (216, 960, 8240), (1805, 36, 1784),
                                   (77, 1580, 9152), (4774, 32, 2904), (524, 1816, 8668), (5383, 320, 4664),
                                   (1314, 3820, 1748), (300, 1084, 8200), (5300, 60, 4600), (1030, 316, 9000)])
def test_wide_tiles(m, n, k):
    """192 and 256 columns with every channel tail, one contraction range and several; sampled rows against fp64."""
    say("wide tiles", m, n, k)
    t = layer(m, n, k, 16)
    ws = torch.full((training.backward_workspace_bytes(m, n, k, 16),), 0xff, dtype=torch.uint8, device=DEV)
    got = run(t, 0.5, workspace=ws, need_lora=False)[0]
    rows = torch.tensor(sorted({0, 1, 15, 16, 63, 64, 255, 256, m // 2, m - 1} & set(range(m))), device=DEV)
    kept = t["kept"]
    part = dict(t, g=t["g"][rows], kept=training.Checkpoint(*(getattr(kept, f)[rows].contiguous()
                                                              for f in ("codes", "exps", "idx", "stats"))))
    ref, tol = reference(part, 0.5)
    check((got[rows], None, None), ref, tol)
