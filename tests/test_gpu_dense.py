"""Dense linears with an epilogue against fp64.

Allowances, U = 2^-24 and H the type's half step: z is off by K + 2 roundings U of the products'
magnitudes; an activation by its steepest slope (1.13) times that and by 2e-5 of itself (the fit
of Phi and the hardware's exponential and reciprocal); a result by H.  Backward, dz enters the
products rounded (H), a sum of n terms is off by n U of their magnitudes."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import dense  # noqa: E402

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24
ACTS = [None, "gelu", "gelu_tanh", "silu"]


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rand(*shape, seed, dtype=BF, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def act64(z, name):
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if name == "silu" else z


def slope64(z, name):
    z = z.clone().requires_grad_()
    return torch.autograd.grad(act64(z, name).sum(), z)[0]


def rows(p, lead):
    """[N] or [batch, N] against [.., N]."""
    return p.double()[:, None] if p.dim() == 2 else p.double()


def check(got, want, allow, what):
    a = allow + half(got.dtype) * 1.01 * (want.abs() + allow) + 2.0 ** -25 * (got.dtype is HF)
    bad = ~((got.double() - want).abs() <= a)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for {float(want[i])}, "
                             f"allowed {float(a[i]):.3g}")


def run(lead, n, k, dtype=BF, act=None, bias=True, gate=None, residual=False, back=False, seed=0):
    x, w = rand(*lead, k, seed=seed, dtype=dtype), rand(n, k, seed=seed + 1, dtype=dtype, std=k ** -0.5)
    b = rand(n, seed=seed + 2, dtype=dtype, std=0.3) if bias else None
    gt = None
    if gate == "sequence":
        gt = rand(lead[0], 3 * n, seed=seed + 3, dtype=dtype)[:, n:2 * n]
    elif gate:
        gt = rand(n, seed=seed + 3, dtype=dtype)
    res = rand(*lead, n, seed=seed + 4, dtype=dtype) if residual else None
    y, z = dense.linear(x, w, b, activation=act, gate=gt, residual=res, keep=True)
    assert torch.equal(dense.linear(x, w, b, activation=act, gate=gt, residual=res), y)
    m = x.numel() // k
    x64, w64 = x.double().reshape(m, k), w.double()
    z64 = torch.mm(x64, w64.t()).view(*lead, n)
    mag = torch.mm(x64.abs(), w64.abs().t()).view(*lead, n)
    if b is not None:
        z64, mag = z64 + b.double(), mag + b.double().abs()
    z_err = (k + 4) * U * mag
    check(z, z64, z_err, "z")
    a = act64(z64, act)
    g64 = torch.ones((), dtype=torch.float64, device=DEV) if gt is None else rows(gt, lead)
    want = a * g64
    err = (1.13 * z_err + (2e-5 * a.abs() if act else 0)) * g64.abs() + 2 * U * want.abs()
    if res is not None:
        want, err = want + res.double(), err + 2 * U * (want.abs() + res.double().abs())
    check(y, want, err, "y")
    if not back:
        return
    dy = rand(*lead, n, seed=seed + 5, dtype=dtype, std=0.5)
    dx, dw, db, dg = dense.linear_backward(dy, x, w, z, activation=act, gate=gt, need_dbias=bias)
    h = half(dtype)
    zk = z.double()
    slope, value = slope64(zk, act), act64(zk, act)
    dz = dy.double() * slope * g64
    # The slope's own error: 2e-5 of its two summands.
    dz_err = (2e-5 * dy.double().abs() * (1 + zk.abs()) * g64.abs() if act else 0) + 4 * U * dz.abs()
    round_ = h if act or gt is not None else 0.0                    # dy itself goes in where nothing changes it
    used = dz_err + round_ * dz.abs() + 2.0 ** -25 * (dtype is HF)
    dz2, used2 = dz.reshape(m, n), used.reshape(m, n)
    check(dx, torch.mm(dz2, w64).view(*lead, k), torch.mm(used2 + (n + 16) * U * dz2.abs(), w64.abs()).view(*lead, k), "dx")
    check(dw, torch.mm(dz2.t(), x64), torch.mm((used2 + (m + 16) * U * dz2.abs()).t(), x64.abs()), "dw")
    if bias:
        check(db, dz2.sum(0), (dz_err.reshape(m, n) + (m + 16) * U * dz2.abs()).sum(0) if act or gt is not None
              else (m + 16) * U * dz2.abs().sum(0), "dbias")
    else:
        assert db is None
    if gt is None:
        assert dg is None
    else:
        per = dy.double() * value
        per_err = 2e-5 * per.abs() + (m + 16) * U * per.abs()
        total = (lambda t: t.sum(1)) if gate == "sequence" else (lambda t: t.reshape(m, n).sum(0))
        check(dg, total(per), total(per_err), "dgate")
        assert dg.shape == gt.shape


SIZES = [(1, 1, 8), (1, 4099, 512), (3, 17, 64), (16, 33, 4096), (16, 16, 40), (17, 64, 72), (32, 130, 1000), (33, 128, 128), (64, 256, 64),
         (100, 1000, 8), (129, 257, 264), (255, 300, 2056), (300, 260, 72), (128, 128, 4096), (512, 768, 200)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sizes(m, n, k, dtype):
    run((m,), n, k, dtype, back=True)
    run((m,), n, k, dtype, act="gelu", gate="shared", residual=True, back=True)


@pytest.mark.parametrize("m,n,k", [(2048, 6400, 136), (2040, 6401, 72), (100, 4096, 3336), (2000, 100, 6664)])
def test_large_tiles(m, n, k):
    """200 tiles of 256 x 256 and more: forward, dw (n x k) and dx (m x k)."""
    run((m,), n, k, act="silu", residual=True, back=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate", [None, "shared", "sequence"])
def test_epilogues(act, gate):
    for residual in (False, True):
        for bias in (False, True):
            run((3, 50), 264, 136, act=act, gate=gate, residual=residual, bias=bias, back=residual)
            run((3, 50), 77, 136, HF, act=act, gate=gate, residual=residual, bias=bias, back=residual)
    run((3, 5), 264, 1544, act=act, gate=gate, residual=True, back=True)


@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_over_their_range(act):
    """The identity times each value: both tails, zeros, the largest."""
    v = torch.cat([torch.linspace(-30, 30, 4001), torch.linspace(-6, 6, 4095), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38]),
                   torch.zeros(2)]).to(BF).to(DEV)
    x = torch.zeros(v.numel(), 8, dtype=BF, device=DEV)
    x[:, 0] = v
    w = torch.eye(8, dtype=BF, device=DEV)
    y, z = dense.linear(x, w, activation=act, keep=True)
    assert torch.equal(z, x)
    x64 = x.double()
    want = act64(x64, act)
    check(y, want, 2e-5 * want.abs() + 1e-37, act)
    g = torch.ones_like(x)
    dx = dense.linear_backward(g, x, w, z, activation=act, need_dw=False)[0]
    slope = slope64(x64.clamp(-1e4, 1e4), act)
    check(dx, slope, 2e-5 * (1 + x64.abs().clamp(max=50)), act + " slope")


def test_into_the_residual():
    x, w, res = rand(2, 300, 64, seed=1), rand(200, 64, seed=2), rand(2, 300, 200, seed=3)
    gate = rand(2, 200, seed=4)
    want = dense.linear(x, w, gate=gate, residual=res)
    got = dense.linear(x, w, gate=gate, residual=res, out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(got, want)
    for m, k in ((4, 512), (70, 4096)):                            # the kernel for few rows; split over k
        x, w, res = rand(m, k, seed=5), rand(72, k, seed=6, std=0.02), rand(m, 72, seed=7)
        want = dense.linear(x, w, residual=res)
        assert torch.equal(dense.linear(x, w, residual=res, out=res), want)


def test_backward_parts():
    x, w, dy = rand(40, 64, seed=1), rand(24, 64, seed=2), rand(40, 24, seed=3)
    z = dense.linear(x, w)
    every = dense.linear_backward(dy, x, w, z, activation="gelu")
    for i, name in enumerate(("need_dx", "need_dw", "need_dbias")):
        flags = {n: n == name for n in ("need_dx", "need_dw", "need_dbias")}
        got = dense.linear_backward(dy, x, w, z, activation="gelu", **flags)
        assert torch.equal(got[i], every[i]) and sum(t is not None for t in got) == 1
    assert all(t is None for t in dense.linear_backward(dy, x, w, z, activation="gelu", need_dx=False, need_dw=False, need_dbias=False))


def test_empty():
    w = rand(24, 64, seed=1)
    e = lambda *s: torch.empty(*s, dtype=BF, device=DEV)  # noqa: E731
    assert dense.linear(e(0, 64), w).shape == (0, 24)
    dx, dw, db, dg = dense.linear_backward(e(2, 0, 24), e(2, 0, 64), w, e(2, 0, 24), activation="gelu", gate=rand(2, 24, seed=2))
    assert dx.shape == (2, 0, 64) and (dw == 0).all() and (db == 0).all() and (dg == 0).all() and dg.shape == (2, 24)
    x = rand(5, 64, seed=3)
    assert dense.linear(x, e(0, 64)).shape == (5, 0)
    dx, dw, db, _ = dense.linear_backward(e(5, 0), x, e(0, 64))
    assert (dx == 0).all() and dw.shape == (0, 64) and db.shape == (0,)


def test_refusals():
    x, w = rand(6, 64, seed=1), rand(24, 64, seed=2)
    b = rand(24, seed=3)
    for bad in (dict(activation="tanh"), dict(bias=b[:8]), dict(gate=rand(6, 24, seed=4)), dict(residual=rand(5, 24, seed=4)),
                dict(out=rand(6, 25, seed=4)), dict(residual=rand(24, 6, seed=4).t()), dict(gate=rand(48, seed=4)[::2])):
        with pytest.raises(ValueError):
            dense.linear(x, w, **bad)
    for bad in (dict(bias=b.half()), dict(gate=b.float()), dict(residual=rand(6, 24, seed=4, dtype=HF)), dict(out=rand(6, 24, seed=1).half())):
        with pytest.raises(TypeError):
            dense.linear(x, w, **bad)
    with pytest.raises(TypeError):
        dense.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        dense.linear(x, w[:, :32].contiguous())
    with pytest.raises(ValueError):
        dense.linear(rand(64, 6, seed=1).t(), w)
    room = rand(7, 64, seed=5)
    with pytest.raises(ValueError):
        dense.linear(room[:6], rand(64, 64, seed=6), out=room[1:])
    with pytest.raises(ValueError):
        dense.linear(x, rand(64, 64, seed=6), residual=room[:6], out=room[1:])
    with pytest.raises(ValueError):
        dense.linear_backward(rand(6, 24, seed=1), x, w, activation="gelu")
    with pytest.raises(ValueError):
        dense.linear_backward(rand(6, 24, seed=1), x, w, gate=b)
    with pytest.raises(ValueError):
        dense.linear_backward(rand(5, 24, seed=1), x, w)
    import activation_sparse_gemm_token_amd as rtl
    with pytest.raises(rtl.RtlError):
        dense.linear(rand(6, 60, seed=1), rand(24, 60, seed=2))    # K % 8
    with pytest.warns(UserWarning, match=r"dense\.linear records no autograd graph"):
        dense.linear(x, w.clone().requires_grad_())


def test_same_bits_and_captured():
    x, w, b, dy = rand(150, 2056, seed=1), rand(130, 2056, seed=2, std=0.02), rand(130, seed=3), rand(150, 130, seed=4)

    def step():
        y, z = dense.linear(x, w, b, activation="gelu", keep=True)
        return (y, z, dense.linear(x[:5], w, b), *dense.linear_backward(dy, x, w, z, activation="gelu")[:3])

    want = step()
    with torch.cuda.stream(torch.cuda.Stream()):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want))
        assert all(torch.equal(a, c) for a, c in zip(step(), want))


@pytest.mark.parametrize("act", ACTS[1:])
def test_a_sum_past_fp32(act):
    """z = inf is its own activation in every form."""
    x = torch.full((40, 8), 3e38, dtype=BF, device=DEV)
    w = torch.ones(16, 8, dtype=BF, device=DEV)
    assert torch.isposinf(dense.linear(x, w, activation=act)).all()


@pytest.mark.parametrize("m,n,k", [(1500, 3000, 3000), (3000, 2701, 2568), (3000, 1001, 5000)])
def test_tiles(m, n, k):
    """Forward, dx and dw in tiles of 256 x 128 and of 256 x 256 each."""
    run((m,), n, k, act="gelu_tanh", gate="shared", residual=True, back=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [64, 65])
def test_a_gate_keeps_z_in_fp32(act, n):
    """One row to a gate row, where nothing averages z's rounding out: dgate is off by the result's half step."""
    x, w, dy = rand(50, 1, 72, seed=1), rand(n, 72, seed=2, std=72 ** -0.5), rand(50, 1, n, seed=3)
    gate = rand(50, n, seed=4)
    y, z = dense.linear(x, w, activation=act, gate=gate, keep=True)
    assert z.dtype is torch.float32
    dg = dense.linear_backward(dy, x, w, z, activation=act, gate=gate)[3]
    z64 = x.double() @ w.double().t()
    want = (dy.double() * act64(z64, act))[:, 0]
    err = 1.13 * (72 + 4) * U * (x.double().abs() @ w.double().t().abs()) + (2e-5 * act64(z64, act).abs() if act else 0)
    check(dg, want, (dy.double().abs() * err)[:, 0] + 2 * U * want.abs(), "dgate")
    rounded = z.to(BF)                                             # is taken too
    dg = dense.linear_backward(dy, x, w, rounded, activation=act, gate=gate)[3]
    want = (dy.double() * act64(rounded.double(), act))[:, 0]
    check(dg, want, 2e-5 * want.abs(), "dgate of a rounded z")


def test_17_to_32_rows_of_a_large_weight():
    """Tiles, the contraction in ranges: a workspace, where 16 rows need none."""
    assert dense.workspace_bytes(30, 12001, 4096) > 0 and dense.workspace_bytes(16, 12001, 4096) == 0
    run((30,), 12001, 4096, act="silu", gate="shared", residual=True)
