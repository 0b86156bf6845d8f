"""The checkpoint with a step of its own for the pruned channels, and the gradients
formed from it: against its definition, against the gradients of the stored values,
and of either form against the gradients of x itself."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import training  # noqa: E402
from workloads import gen  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_gpu_training_forms as forms  # noqa: E402
import train_plain as plain  # noqa: E402
from fine_plain import pack_fine, select, values_fine  # noqa: E402

DEV = "cuda:0"
FIELDS = ("codes", "exps", "pruned_exps", "idx", "stats")


def say(*a):
    print("[fine]", *a, file=sys.stderr, flush=True)


def to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def inputs(m, k, law, seed):
    rng = np.random.default_rng(seed)
    if law == "mixture":
        return gen.mixture_bernoulli(rng, m, k)
    if law == "ties":
        return gen.tie_heavy(rng, m, k)
    if law == "gelu":
        return gen.gelu_of_normal(rng, m, k)
    bits = gen.uniform_bits(rng, (m, k), emax=100, span=220)
    bits[::3, :k // 2] = 0
    bits[1::5] &= 0x807f                                           # subnormal rows
    return bits


@pytest.mark.parametrize("law", ["mixture", "ties", "gelu", "wild"])
@pytest.mark.parametrize("m,k", [(1, 4), (1, 8), (3, 12), (5, 32), (2, 36), (7, 68), (4, 512), (33, 516), (9, 1024),
                                 (300, 1028), (130, 2056), (6, 12288), (9000, 64), (1, 12292)])
def test_it_is_the_defined_one(m, k, law):
    say(m, k, law)
    x = to_dev(inputs(m, k, law, m + k))
    kept, one = training.checkpoint(x, fine=True), training.checkpoint(x)
    v = plain.bf16(x)
    mk = select(v)
    codes, exps, pruned = pack_fine(v, mk)
    assert np.array_equal(kept.codes.cpu().numpy(), codes)
    assert np.array_equal(kept.exps.cpu().numpy(), exps) and np.array_equal(kept.pruned_exps.cpu().numpy(), pruned)
    for n in ("exps", "idx", "stats"):                             # what both forms hold is the same
        assert torch.equal(getattr(kept, n), getattr(one, n)), n
    at = torch.from_numpy(mk).to(DEV) == 1
    assert torch.equal(kept.codes[at], one.codes[at]) and one.pruned_exps is None
    stored = values_fine(codes, exps, pruned, mk)
    assert np.array_equal(plain.bf16(kept.unpack()), stored)
    out = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    assert kept.unpack(out=out).data_ptr() == out.data_ptr() and np.array_equal(plain.bf16(out), stored)
    step = np.repeat(2.0 ** (pruned.astype(float) - 133), 32, 1)[:, :k]
    assert (np.abs(stored - v) <= np.where(np.abs(v) < step / 2, step, step / 2))[mk == 0].all()
    assert np.array_equal(np.sign(stored)[mk == 0], np.sign(v)[mk == 0])


def test_it_writes_only_its_rows():
    for m, k in ((3, 36), (5, 520), (2, 4)):
        x = to_dev(inputs(m, k, "mixture", 4))
        want = training.checkpoint(x, fine=True)
        guard, views = {}, {}
        for name in FIELDS:
            w = getattr(want, name)
            guard[name] = torch.full((w.numel() + 256,), 77, dtype=w.dtype, device=DEV)
            views[name] = guard[name][128:128 + w.numel()]
        assert training._fn("rtl_checkpoint_pack_fine")(x.data_ptr(), m, k, *[views[n].data_ptr() for n in FIELDS], None) == 0
        y = torch.full((m * k + 256,), 77, dtype=torch.bfloat16, device=DEV)
        assert training._fn("rtl_checkpoint_unpack_fine")(*[views[n].data_ptr() for n in FIELDS[:4]], m, k,
                                                          y[128:].data_ptr(), None) == 0
        torch.cuda.synchronize()
        for name, buf in guard.items():
            n = views[name].numel()
            assert (buf[:128] == 77).all() and (buf[128 + n:] == 77).all(), name
            assert torch.equal(views[name], getattr(want, name).flatten()), name
        assert (y[:128] == 77).all() and (y[128 + m * k:] == 77).all()
        assert torch.equal(y[128:128 + m * k].view(m, k), want.unpack())


def test_rows_without_anything_and_not_finite_ones():
    x = to_dev(inputs(8, 128, "mixture", 3))
    x[1] = 0
    want = training.checkpoint(x, fine=True)
    assert (want.unpack()[1] == 0).all() and (want.pruned_exps[1] == 0).all()
    x[2, 17], x[5, 99] = float("inf"), float("nan")
    got = training.checkpoint(x, fine=True)
    rows = [0, 1, 3, 4, 6, 7]
    for n in FIELDS:
        assert torch.equal(getattr(got, n)[rows], getattr(want, n)[rows])
    empty = training.checkpoint(torch.empty(0, 3, 64, dtype=torch.bfloat16, device=DEV), fine=True)
    assert empty.unpack().shape == (0, 3, 64)


def layer(m, n, k, r, law="mixture", fine=True):
    g = torch.Generator().manual_seed(m + n + k + r)
    rand = lambda std, *s: (std * torch.randn(*s, generator=g)).bfloat16().to(DEV)  # noqa: E731
    x = to_dev(inputs(m, k, law, m + k))
    return dict(x=x, kept=training.checkpoint(x, fine=fine), g=rand(0.01, m, n), w_t=rand(0.02, k, n), a=rand(0.05, r, k),
                b=rand(0.05, n, r))


def run(d, alpha, **kw):
    return training.sparse_linear_backward(d["g"], d["kept"], d["w_t"], d["a"], d["b"], alpha, **kw)


def outside(got, want, tol):
    return [n for n, y, w, e in zip(("dx", "da", "db"), got, want, tol) if not bool(((y.double() - w).abs() <= e).all())]


@pytest.mark.parametrize("law", ["mixture", "gelu", "ties"])
@pytest.mark.parametrize("m,n,k,r", [(1, 4, 4, 1), (3, 12, 20, 5), (33, 100, 36, 32), (64, 128, 256, 33), (77, 264, 520, 16),
                                     (77, 260, 516, 64), (130, 520, 1028, 100), (300, 132, 2052, 64), (414, 32, 7304, 16),
                                     (520, 1392, 8884, 16), (1246, 524, 1660, 8), (2050, 6404, 3108, 64), (1300, 2404, 3112, 128)])
def test_gradients_of_the_stored_values(m, n, k, r, law):
    say(m, n, k, r, law)
    d = layer(m, n, k, r, law)
    ws = torch.full((training.backward_workspace_bytes(m, n, k, r),), 0xff, dtype=torch.uint8, device=DEV)
    got = run(d, -0.75, workspace=ws)
    assert outside(got, *forms.reference(d, -0.75)) == []
    for p, q in zip(got, run(d, -0.75)):
        assert torch.equal(p, q)


def gradients(x, kept, d, alpha):
    """The formulas in fp64 at the values x."""
    k = x.shape[1]
    g, w, a, b = (d[i].double() for i in ("g", "w_t", "a", "b"))
    mk, s, lk = forms.mask(kept.idx, k), kept.stats[:, :1].double(), kept.stats[:, 1:].double()
    u = alpha * (g @ b)
    v = u @ a
    e = g @ forms.t(w) - v
    share = torch.where(lk > 0, (mk * x * e).sum(1, keepdim=True) / lk, 0.0)
    rest = x * (1 - s * mk)
    return (v + s * mk * e + share * torch.sign(x) * (1 - s * mk), forms.t(u) @ rest,
            forms.t(g) @ (alpha * (rest @ forms.t(a)))), u, e, share, mk, s, lk


@pytest.mark.parametrize("law", ["mixture", "gelu"])
@pytest.mark.parametrize("fine", [False, True])
@pytest.mark.parametrize("m,n,k,r", [(77, 264, 520, 16), (300, 516, 1028, 64)])
def test_gradients_of_x_itself(m, n, k, r, fine, law):
    """Each gradient is off by what the codes' own error makes of it (half a step, or
    one step for a pruned value below half of one; a lost sign) and the kernels'
    tolerance, element by element."""
    say(m, n, k, r, fine, law)
    alpha = 0.75
    d = layer(m, n, k, r, law, fine)
    kept, x = d["kept"], d["x"].double()
    stored = kept.unpack().double()
    (want, u, e, share, mk, s, lk) = gradients(x, kept, d, alpha)
    got = run(d, alpha)
    _, tol = forms.reference(d, alpha)

    step = lambda e: torch.from_numpy(np.repeat(2.0 ** (plain.bf16(e) - 133), 32, 1)[:, :k]).to(DEV)  # noqa: E731
    err = step(kept.exps) / 2
    if fine:
        p = step(kept.pruned_exps)
        err = torch.where(mk == 1, err, torch.where(x.abs() < p / 2, p, p / 2))
    assert bool(((stored - x).abs() <= err).all())
    turn, (a, b, g) = (1 - s * mk).abs(), (d[i].double().abs() for i in ("a", "b", "g"))
    lost = torch.sign(stored) != torch.sign(x)
    if fine:
        assert not bool((lost & (mk == 0)).any())
    share_off = torch.where(lk > 0, (mk * err * e.abs()).sum(1, keepdim=True) / lk, 0.0)
    off = (turn * (share_off + lost * (share.abs() + share_off)), forms.t(u.abs()) @ (turn * err),
           forms.t(g) @ (abs(alpha) * ((turn * err) @ forms.t(a))))
    # the kernels' tolerance has half a step of the stored values' result; of this one's, that of the distance more
    assert outside(got, want, [t + o * (1 + plain.HALF_BF16) for t, o in zip(tol, off)]) == []
    if law == "mixture":
        rel = [((y.double() - w).norm() / w.norm()).item() for y, w in zip(got, want)]
        say("relative error of dx, da, db against x's own:", rel)
        assert max(rel[1:]) < 0.03 if fine else min(rel[1:]) > 0.1


def test_captured_on_two_streams_and_without_parts():
    m, n, k, r = 130, 264, 520, 16
    d = layer(m, n, k, r)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = training.checkpoint(d["x"], fine=True)
        outs = (*training.sparse_linear_backward(d["g"], kept, d["w_t"], d["a"], d["b"]), kept.unpack())
    for i in range(4):
        d["x"].copy_(to_dev(inputs(m, k, "mixture", 20 + i)))
        now = training.checkpoint(d["x"], fine=True)
        eager = (*training.sparse_linear_backward(d["g"], now, d["w_t"], d["a"], d["b"]), now.unpack())
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(outs, eager):
            assert torch.equal(p, q)
    d["kept"] = now
    dx, da, db = run(d, 1.0)
    only = run(d, 1.0, need_lora=False)
    assert torch.equal(only[0], dx) and only[1] is None
    lora = run(d, 1.0, need_dx=False)
    assert lora[0] is None and torch.equal(lora[1], da) and torch.equal(lora[2], db)
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            res.append(run(d, 1.0))
    torch.cuda.synchronize()
    for out in res:
        assert all(torch.equal(p, q) for p, q in zip(out, (dx, da, db)))


def test_refusals():
    kept = training.checkpoint(to_dev(inputs(8, 128, "mixture", 1)), fine=True)
    args = (kept.codes, kept.exps, kept.idx, kept.stats)
    for bad, what in ((kept.pruned_exps.int(), TypeError), (kept.pruned_exps[:, :3].contiguous(), ValueError),
                      (kept.pruned_exps.cpu(), ValueError), (kept.pruned_exps.t().contiguous().t(), ValueError)):
        with pytest.raises(what):
            training.Checkpoint(*args, pruned_exps=bad)
    again = training.Checkpoint(*args, lead=(2, 4), pruned_exps=kept.pruned_exps)
    assert torch.equal(again.unpack(), kept.unpack().view(2, 4, 128))
    with pytest.raises(ValueError):
        kept.unpack(out=torch.empty(8, 124, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        training.checkpoint(torch.zeros(8, 128, device=DEV), fine=True)
    with pytest.raises(rtl.RtlError) as e:
        training.checkpoint(torch.zeros(8, 126, dtype=torch.bfloat16, device=DEV), fine=True)
    assert e.value.status == 2
