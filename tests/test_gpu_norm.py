"""Layer norm against fp64.

Allowances, U = 2^-24 (fp32's half step) and H the type's: a thread adds at most 32 values in
a row, then 6 levels of lanes and up to 16 wavefronts, so a sum is off by 60 U of its
magnitudes; the mean so; the variance and rstd relative to themselves; a result by H."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import norm  # noqa: E402

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24
K = 60 * U


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rand(*shape, seed, dtype=F32, std=1.0, mean=0.0):
    return (mean + std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def rows_of(p, x):
    """[C] or [batch, C] against x [batch, tokens, C] (or fewer dimensions)."""
    return p.double()[:, None] if p.dim() == 2 else p.double()


def normalised(x, eps):
    """(xhat, its allowance, mean, rstd, allowance of the mean) in fp64."""
    v = x.double()
    mean = v.mean(-1, keepdim=True)
    c = v - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    m_err = K * v.abs().mean(-1, keepdim=True)
    # The mean's error moves every value, and the variance by its square; the centred values
    # are off by U of themselves, the variance by K of itself more.
    r_rel = K + (m_err * rstd) ** 2 + 4 * U
    return c * rstd, (m_err + U * c.abs()) * rstd + (r_rel + 4 * U) * (c * rstd).abs(), mean, rstd, m_err, r_rel


def forward_want(x, w, b, eps, offset):
    xhat, err, *_ = normalised(x, eps)
    f = torch.ones((), dtype=torch.float64, device=DEV) if w is None else rows_of(w, x) + offset
    y = xhat * f
    allow = err * f.abs() + 4 * U * y.abs()
    if b is not None:
        y = y + rows_of(b, x)
        allow = allow + 2 * U * y.abs()
    return y, allow


def check(got, want, allow, what):
    a = allow + half(got.dtype) * 1.01 * (want.abs() + allow) + 2.0 ** -25 * (got.dtype is HF)
    bad = ~((got.double() - want).abs() <= a)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for {float(want[i])}, "
                             f"allowed {float(a[i]):.3g}")


def backward_want(dy, x, w, eps, offset):
    xhat, xe, mean, rstd, m_err, r_rel = normalised(x, eps)
    d = dy.double()
    f = torch.ones((), dtype=torch.float64, device=DEV) if w is None else rows_of(w, x) + offset
    g = d * f
    s1, s2 = (g * xhat).mean(-1, keepdim=True), g.mean(-1, keepdim=True)
    dx = rstd * (g - s2 - xhat * s1)
    ge = 2 * U * g.abs()
    s1e = K * (g * xhat).abs().mean(-1, keepdim=True) + (g.abs() * xe).mean(-1, keepdim=True)
    s2e = K * g.abs().mean(-1, keepdim=True)
    dx_allow = rstd * (ge + s2e + xe * s1.abs() + xhat.abs() * s1e + 4 * U * (g.abs() + s2.abs() + (xhat * s1).abs())) + \
        (r_rel + 4 * U) * dx.abs()
    return dx, dx_allow, d * xhat, (d.abs() * xe)


def run(shape, dtype, affine, offset=0.0, eps=1e-5, wtype=None, std=1.0, mean=0.3, seed=0):
    c = shape[-1]
    x, dy = rand(*shape, seed=seed, dtype=dtype, std=std, mean=mean), rand(*shape, seed=seed + 1, dtype=dtype, std=0.5)
    w = b = None
    if affine:
        rows = (shape[0], c) if affine == "sequence" else (c,)
        w, b = (rand(*rows, seed=seed + i, dtype=wtype or dtype, std=0.3) for i in (2, 3))
    y, m, r = norm.layer_norm(x, w, b, eps=eps, offset=offset, return_stats=True)
    check(y, *forward_want(x, w, b, eps, offset), "y")
    xhat, xe, mean64, rstd64, m_err, r_rel = normalised(x, eps)
    check(m, mean64[..., 0], m_err[..., 0] + U * mean64[..., 0].abs(), "mean")
    check(r, rstd64[..., 0], (r_rel + 4 * U)[..., 0] * rstd64[..., 0], "rstd")
    assert torch.equal(norm.layer_norm(x, w, b, eps=eps, offset=offset), y)
    dx, dw, db = norm.layer_norm_backward(dy, x, m, r, w, offset=offset)
    dx64, allow, per, per_err = backward_want(dy, x, w, eps, offset)
    check(dx, dx64, allow, "dx")
    if not affine:
        assert dw is None and db is None
        return
    total = lambda t: t.sum(1) if affine == "sequence" else t.reshape(-1, c).sum(0)  # noqa: E731
    n = x.numel() // c
    # A thread adds up to n / 256 + 1 rows one by one, then sets of rows and parts.
    ks = (n / 256 + 1 + 16 + 16 + 16 + 4) * U
    d64 = dy.double()
    check(dw, total(per), total(per_err + ks * per.abs()), "dweight")
    check(db, total(d64), ks * total(d64.abs()), "dbias")
    only = norm.layer_norm_backward(dy, x, m, r, w, offset=offset, need_affine=False)
    assert torch.equal(only[0], dx) and only[1] is None
    only = norm.layer_norm_backward(dy, x, m, r, w, offset=offset, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dw) and torch.equal(only[2], db)


CHANNELS = [1, 2, 7, 8, 63, 64, 65, 100, 128, 129, 200, 256, 260, 512, 520, 1023, 1024, 1028, 2048, 2052, 2049, 4096, 4100, 5001, 8192, 8200, 12288, 16384,
            16392, 20001, 32768]


@pytest.mark.parametrize("c", CHANNELS)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_channels(c, dtype):
    run((3, 7, c), dtype, "shared")


@pytest.mark.parametrize("affine", [None, "shared", "sequence"])
@pytest.mark.parametrize("wtype", [None, F32])
@pytest.mark.parametrize("shape", [(1, 1, 96), (2, 300, 96), (5, 33, 1028), (1, 1500, 640), (3, 70, 4104), (2, 5, 9001)])
def test_affine(shape, affine, wtype):
    for dtype in (BF, F32):
        run(shape, dtype, affine, offset=1.0, wtype=wtype)


@pytest.mark.parametrize("shape", [(64,), (5, 64), (2, 3, 4, 64)])
def test_dimensions(shape):
    run(shape, BF, "shared")


@pytest.mark.parametrize("std,mean", [(1.0, 1000.0), (1e-3, 5.0), (1e-20, 0.0), (300.0, 0.0)])
def test_magnitudes(std, mean):
    """A mean far from zero: the variance is that of the centred values."""
    run((2, 9, 1000), F32, "shared", std=std, mean=mean)


def test_a_constant_row():
    x = torch.full((3, 4, 256), 2.5, device=DEV, dtype=BF)
    y, m, r = norm.layer_norm(x, return_stats=True)
    assert (y == 0).all() and (m == 2.5).all()
    assert ((r.double() - 1e-5 ** -0.5).abs() <= 8 * U * 1e-5 ** -0.5).all()


def test_strides_and_in_place():
    """A part of the tokens, slices of a modulation row, rows that are only 2-byte aligned, in place."""
    joint, rows = rand(2, 50, 136, seed=1, dtype=BF), rand(2, 6 * 136, seed=2, dtype=BF)
    x, w, b = joint[:, 7:30], rows[:, 136:272], rows[:, 272:408]
    want = norm.layer_norm(x.contiguous(), w.contiguous(), b.contiguous(), offset=1.0, return_stats=True)
    got = norm.layer_norm(x, w, b, offset=1.0, return_stats=True)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    dy = rand(2, 60, 136, seed=3, dtype=BF)[:, 3:26]
    grads = norm.layer_norm_backward(dy, x, got[1], got[2], w, offset=1.0)
    again = norm.layer_norm_backward(dy.contiguous(), x.contiguous(), got[1], got[2], w.contiguous(), offset=1.0)
    assert all(torch.equal(a, c) for a, c in zip(grads, again))
    odd = rand(3, 41, 40, seed=4, dtype=BF)[:, :, 1:38]
    check(norm.layer_norm(odd), *forward_want(odd, None, None, 1e-5, 0.0), "odd rows")
    before = joint.clone()
    y = norm.layer_norm(x, w, b, offset=1.0, out=x)
    assert y.data_ptr() == x.data_ptr() and torch.equal(y, want[0])
    assert torch.equal(joint[:, :7], before[:, :7]) and torch.equal(joint[:, 30:], before[:, 30:])
    out = torch.zeros_like(before)
    norm.layer_norm(before[:, 7:30], w, b, offset=1.0, out=out[:, 7:30])
    assert torch.equal(out[:, 7:30], want[0]) and (out[:, :7] == 0).all() and (out[:, 30:] == 0).all()
    one = rand(1, 1, 64, seed=5, dtype=BF).expand(3, 5, 64)
    assert torch.equal(norm.layer_norm(one), norm.layer_norm(one.contiguous()))


def test_refusals():
    x, w = rand(2, 3, 64, seed=1, dtype=BF), rand(64, seed=2, dtype=BF)
    stats = norm.layer_norm(x, return_stats=True)[1:]
    for bad in (dict(bias=w), dict(weight=w[:32]), dict(weight=rand(3, 64, seed=1, dtype=BF)), dict(out=x[:, :2]),
                dict(out=x.as_strided((2, 3, 64), (64, 64, 1))), dict(weight=w, out=torch.empty(2, 3, 32, dtype=BF, device=DEV)),
                dict(weight=w, bias=rand(64, seed=3)[None].expand(2, 64)[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            norm.layer_norm(x, **bad)
    for bad in (dict(weight=w.half()), dict(weight=w, bias=w.float()), dict(out=x.half())):
        with pytest.raises(TypeError):
            norm.layer_norm(x, **bad)
    room = rand(3, 3, 64, seed=4, dtype=BF)
    with pytest.raises(ValueError):
        norm.layer_norm(room[:2], out=room[1:])
    with pytest.raises(ValueError):
        norm.layer_norm(x.transpose(1, 2))
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x[:1], x, *stats)
    with pytest.raises(TypeError):
        norm.layer_norm_backward(x.float(), x, *stats)
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x, x, stats[0][:1], stats[1])
    with pytest.raises(ValueError):
        norm.layer_norm_backward(x, x, stats[0].double(), stats[1])
    with pytest.warns(UserWarning, match=r"norm\.layer_norm records no autograd graph"):
        norm.layer_norm(x, w.clone().requires_grad_())


def test_empty():
    w = rand(2, 64, seed=1, dtype=BF)
    x = torch.empty(2, 0, 64, dtype=BF, device=DEV)
    y, m, r = norm.layer_norm(x, w, w, return_stats=True)
    assert y.shape == x.shape and m.shape == (2, 0)
    dx, dw, db = norm.layer_norm_backward(x, x, m, r, w)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
    none = torch.empty(0, 5, 64, dtype=BF, device=DEV)
    y, m, r = norm.layer_norm(none, w[0], w[0], return_stats=True)
    dx, dw, db = norm.layer_norm_backward(none, none, m, r, w[0])
    assert (dw == 0).all() and dw.shape == (64,)
    dx, dw, db = norm.layer_norm_backward(none, none, m, r, w[:0])
    assert dw.shape == (0, 64)


def test_same_bits_and_captured():
    x, dy, w = rand(4, 600, 1032, seed=1, dtype=BF), rand(4, 600, 1032, seed=2, dtype=BF), rand(4, 1032, seed=3, dtype=BF)

    def step():
        y, m, r = norm.layer_norm(x, w, w, offset=1.0, return_stats=True)
        return (y, *norm.layer_norm_backward(dy, x, m, r, w, offset=1.0))

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
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_fp32_weights_on_half_their_access():
    """fp32 weight and bias that begin 8 bytes past a multiple of 16, beside bf16 rows."""
    x, dy = rand(3, 40, 96, seed=1, dtype=BF), rand(3, 40, 96, seed=2, dtype=BF)
    w, b = (rand(3, 98, seed=i)[:, 2:] for i in (3, 4))
    assert w.data_ptr() % 16 == 8
    y, m, r = norm.layer_norm(x, w, b, return_stats=True)
    check(y, *forward_want(x, w, b, 1e-5, 0.0), "y")
    dx = norm.layer_norm_backward(dy, x, m, r, w)[0]
    check(dx, *backward_want(dy, x, w, 1e-5, 0.0)[:2], "dx")


def test_weights_of_many_sequences():
    """More sequences with rows of their own than a grid's second dimension holds."""
    run((70_000, 1, 16), BF, "sequence", seed=5)
