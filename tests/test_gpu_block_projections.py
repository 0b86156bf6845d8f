"""The projections of a block as they are used together.

Serving: a row of modulation from a 4-bit linear, Q and K from one prepared
activation, both rotated.  Training: the input kept in 8 bits, the projection,
the rotation, and back through both to the gradients of x, A and B.  Each step
is checked against fp64 on what it was given, and the whole training step
against fp64 with every rounding on the way counted."""
import os
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
from activation_sparse_gemm_token_amd import rotary, training, w4  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_plain as plain  # noqa: E402

DEV = "cuda:0"
B, T, H, D = 2, 96, 4, 32                                # batch, tokens, heads, head channels
M, K, N, R = B * T, 256, H * D, 16
SECTIONS = [2, 6, 8]


def to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def rand(shape, seed, std):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).bfloat16().to(DEV)


def block(seed):
    rng = np.random.default_rng(seed)
    return dict(x=to_dev(gen.mixture_bernoulli(rng, M, K)), w=rand((N, K), seed + 1, 0.02), a=rand((R, K), seed + 2, 0.05),
                b=rand((N, R), seed + 3, 0.05), freq=rotary.frequencies(D).to(DEV),
                pos=torch.randint(0, 64, (B, T, 3), generator=torch.Generator().manual_seed(seed)).to(DEV))


def turned(v, pos, freq, inverse=False):
    """fp64 rotation (interleaved pairs) of [B, T, H, D]."""
    axis = np.repeat(np.arange(3), SECTIONS)
    ang = pos.cpu().numpy().astype(float)[..., axis] * freq.cpu().numpy()
    z = np.exp((-1j if inverse else 1j) * ang)[:, :, None]
    c = (v[..., 0::2] + 1j * v[..., 1::2]) * z
    out = np.empty_like(v)
    out[..., 0::2], out[..., 1::2] = c.real, c.imag
    return out


def test_serving_step():
    t = block(1)
    wk = rand((N, K), 9, 0.02)
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 256, (2 * K, 64), generator=g, dtype=torch.uint8).to(DEV)
    scales = (0.01 * torch.rand(2 * K, 1, generator=g) + 0.001).bfloat16().to(DEV)
    weight = w4.pack(codes, scales)
    cond = rand((B, 128), 4, 1.0)
    mod = w4.linear(cond, weight)                          # shift and scale of both images
    shift, scale = mod.view(B, 1, 2, K).unbind(2)
    x = (t["x"].view(B, T, K) * (1 + scale) + shift).contiguous()
    prep = rtl.prepare(x)
    q, k = rtl.apply(prep, t["w"]).view(B, T, H, D), rtl.apply(prep, wk).view(B, T, H, D)
    qr, kr = rotary.rope(q, t["pos"], t["freq"], k=k, layout="interleaved", sections=SECTIONS)
    torch.cuda.synchronize()
    for y, v, w in ((qr, q, t["w"]), (kr, k, wk)):
        ref = oracle.sparse_linear_ref(x.view(M, K).contiguous().view(torch.int16).cpu().numpy().view(np.uint16),
                                       w.view(torch.int16).cpu().numpy().view(np.uint16), None, None, 1.0)
        got = plain.bf16(v).reshape(M, N)
        assert (np.abs(got - ref) <= 1e-2 * np.abs(ref) + 1e-3 * np.sqrt(np.mean(ref ** 2))).all()
        want = turned(plain.bf16(v), t["pos"], t["freq"])
        mag = np.repeat(np.abs(plain.bf16(v)[..., 0::2]) + np.abs(plain.bf16(v)[..., 1::2]), 2, -1)
        assert (np.abs(plain.bf16(y) - want) <= 2.0 ** -8 * np.abs(want) + 8 * 2.0 ** -24 * mag).all()
    # in place, queries and keys of one fused tensor: the same numbers
    fused = torch.cat([q, k], 2).contiguous()
    rotary.rope(fused[:, :, :H], t["pos"], t["freq"], k=fused[:, :, H:], layout="interleaved", sections=SECTIONS,
                out=fused[:, :, :H], k_out=fused[:, :, H:])
    assert torch.equal(fused[:, :, :H], qr) and torch.equal(fused[:, :, H:], kr)


def train_step(t, w_t, dy):
    kept = training.checkpoint(t["x"])
    q = rtl.sparse_linear(t["x"], t["w"], t["a"], t["b"], 0.5).view(B, T, H, D)
    y = rotary.rope(q, t["pos"], t["freq"], layout="interleaved", sections=SECTIONS)
    dq = rotary.rope_backward(dy, t["pos"], t["freq"], layout="interleaved", sections=SECTIONS)
    dx, da, db = training.sparse_linear_backward(dq.view(M, N), kept, w_t, t["a"], t["b"], 0.5)
    return kept, y, dq, dx, da, db


def test_training_step():
    t = block(2)
    w_t = t["w"].t().contiguous()
    dy = rand((B, T, H, D), 5, 0.01)
    kept, y, dq, dx, da, db = train_step(t, w_t, dy)
    torch.cuda.synchronize()
    exact_dq = turned(plain.bf16(dy), t["pos"], t["freq"], inverse=True).reshape(M, N)
    mag = np.repeat(np.abs(plain.bf16(dy)[..., 0::2]) + np.abs(plain.bf16(dy)[..., 1::2]), 2, -1).reshape(M, N)
    off = 2.0 ** -8 * np.abs(exact_dq) + 8 * 2.0 ** -24 * mag          # of dq
    assert (np.abs(plain.bf16(dq).reshape(M, N) - exact_dq) <= off).all()
    x = plain.values(kept.codes.cpu().numpy(), kept.exps.cpu().numpy())
    mk = plain.mask(kept.idx.cpu().numpy(), K)
    s, lk = kept.stats.cpu().double().numpy().T
    args = (x, mk, s, lk, plain.bf16(w_t), plain.bf16(t["a"]), plain.bf16(t["b"]), 0.5)
    ref, tol = plain.backward(exact_dq, *args)
    # The gradients are linear in dq: its rounding moves them by at most what
    # |dq's error| gives with every factor's magnitude.
    A, Bm, X = np.abs(plain.bf16(t["a"])), np.abs(plain.bf16(t["b"])), np.abs(x)
    du = 0.5 * off @ Bm
    de = off @ np.abs(plain.bf16(t["w"])) + du @ A
    dd = (mk * X * de).sum(1, keepdims=True) / np.where(lk > 0, lk, 1)[:, None]
    turn = np.abs(1 - s[:, None] * mk)
    rest = X * turn
    moved = (turn * (du @ A) + s[:, None] * mk * (off @ np.abs(plain.bf16(t["w"]))) + dd * turn, du.T @ rest,
             off.T @ (0.5 * rest @ A.T))
    for name, got, want, a, b in zip(("dx", "da", "db"), (dx, da, db), ref, tol, moved):
        d = np.abs(plain.bf16(got) - want)
        # the second half step: the gradient of the rounded dq is rounded, not that of the exact one
        assert (d <= a + b * (1 + 2.0 ** -8)).all(), f"{name}: worst {(d - a - b).max()}"
    assert torch.isfinite(y.float()).all()


def test_training_step_captured_and_replayed():
    t = block(3)
    w_t = t["w"].t().contiguous()
    dy = rand((B, T, H, D), 6, 0.01)
    train_step(t, w_t, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = train_step(t, w_t, dy)
    for i in range(4):
        t["x"].copy_(to_dev(gen.mixture_bernoulli(np.random.default_rng(30 + i), M, K)))
        dy.copy_(rand((B, T, H, D), 40 + i, 0.01))
        eager = train_step(t, w_t, dy)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held[1:], eager[1:]):
            assert torch.equal(a, b)
        assert torch.equal(held[0].codes, eager[0].codes) and torch.equal(held[0].idx, eager[0].idx)


def test_two_streams_at_once():
    steps = [block(10), block(20)]
    dys = [rand((B, T, H, D), 7, 0.01), rand((B, T, H, D), 8, 0.01)]
    w_ts = [t["w"].t().contiguous() for t in steps]
    want = [train_step(t, w, g) for t, w, g in zip(steps, w_ts, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, t, w, g in zip(streams, steps, w_ts, dys):
        with torch.cuda.stream(s):
            got.append(train_step(t, w, g))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for p, q in zip(a[1:], b[1:]):
            assert torch.equal(p, q)
