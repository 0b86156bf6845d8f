"""A transformer block of the operators together, forward and backward: layer norm with a modulation
row, the Q/K/V projection, rotary positions, attention over packed sequences, the output projection into the
gated residual stream, and the MLP likewise.  Every step is checked against fp64 on what it was given; the
step as a whole inside autograd, captured, and on another stream gives the same bits."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import attention, dense, norm, rotary, w4  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import attn_plain  # noqa: E402
import test_gpu_dense as on_dense  # noqa: E402
import test_gpu_norm as on_norm  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16
B, T, C, HQ, HK, D, F = 2, 150, 256, 4, 2, 64, 520            # sequences, tokens, channels, heads, MLP channels
EPS = 1e-5


def rand(*s, seed, std=1.0):
    return (std * torch.randn(*s, generator=torch.Generator().manual_seed(seed))).to(BF).to(DEV)


def weights(seed):
    n = C + (HQ + 2 * HK) * D
    return dict(qkv=rand((HQ + 2 * HK) * D, C, seed=seed, std=C ** -0.5), out=rand(C, HQ * D, seed=seed + 1, std=0.06),
                up=rand(F, C, seed=seed + 2, std=C ** -0.5), down=rand(C, F, seed=seed + 3, std=F ** -0.5),
                b_qkv=rand(n - C, seed=seed + 4, std=0.1), b_up=rand(F, seed=seed + 5, std=0.1), b_down=rand(C, seed=seed + 6, std=0.1))


class Attend(torch.autograd.Function):
    """How a model uses the attention in training (the other operators likewise)."""

    @staticmethod
    def forward(ctx, q, k, v, starts):
        o, lse = attention.attention(q, k, v, causal=True, q_starts=starts, return_lse=True)
        ctx.save_for_backward(q, k, v, o, lse, starts)
        return o

    @staticmethod
    def backward(ctx, g):
        q, k, v, o, lse, starts = ctx.saved_tensors
        return (*attention.attention_backward(g, q, k, v, o, lse, causal=True, q_starts=starts), None)


def forward(x, mod, w, pos, freq, starts):
    """x [B, T, C], mod [B, 6 C]: the block's output and everything on the way."""
    s = dict(x=x)
    sh1, sc1, g1, sh2, sc2, g2 = mod.chunk(6, -1)
    s["h1"], s["m1"], s["r1"] = norm.layer_norm(x, sc1, sh1, offset=1.0, return_stats=True)
    s["qkv"], s["z_qkv"] = dense.linear(s["h1"], w["qkv"], w["b_qkv"], keep=True)
    qkv = s["qkv"].view(B * T, HQ + 2 * HK, D)
    s["q"], s["k"] = rotary.rope(qkv[:, :HQ], pos, freq, k=qkv[:, HQ:HQ + HK])
    s["v"] = qkv[:, HQ + HK:]
    s["o"], s["lse"] = attention.attention(s["q"], s["k"], s["v"], causal=True, q_starts=starts, return_lse=True)
    s["x1"], s["z_out"] = dense.linear(s["o"].view(B, T, HQ * D), w["out"], gate=g1, residual=x, keep=True)
    s["h2"], s["m2"], s["r2"] = norm.layer_norm(s["x1"], sc2, sh2, offset=1.0, return_stats=True)
    s["a"], s["z_up"] = dense.linear(s["h2"], w["up"], w["b_up"], activation="gelu_tanh", keep=True)
    s["y"], s["z_down"] = dense.linear(s["a"], w["down"], w["b_down"], gate=g2, residual=s["x1"], keep=True)
    return s


def backward(dy, s, mod, w, pos, freq, starts):
    sh1, sc1, g1, sh2, sc2, g2 = mod.chunk(6, -1)
    d = dict(dy=dy)
    d["a"], d["w_down"], d["b_down"], d["g2"] = dense.linear_backward(dy, s["a"], w["down"], s["z_down"], gate=g2)
    d["h2"], d["w_up"], d["b_up"], _ = dense.linear_backward(d["a"], s["h2"], w["up"], s["z_up"], activation="gelu_tanh")
    d["n2"], d["sc2"], d["sh2"] = norm.layer_norm_backward(d["h2"], s["x1"], s["m2"], s["r2"], sc2, offset=1.0)
    d["x1"] = dy + d["n2"]
    d["o"], d["w_out"], _, d["g1"] = dense.linear_backward(d["x1"], s["o"].view(B, T, HQ * D), w["out"], s["z_out"], gate=g1,
                                                          need_dbias=False)
    d["q"], d["k"], d["v"] = attention.attention_backward(d["o"].view(B * T, HQ, D), s["q"], s["k"], s["v"], s["o"], s["lse"],
                                                         causal=True, q_starts=starts)
    dqkv = torch.empty(B * T, HQ + 2 * HK, D, dtype=BF, device=DEV)
    rotary.rope_backward(d["q"], pos, freq, k=d["k"], out=dqkv[:, :HQ], k_out=dqkv[:, HQ:HQ + HK])
    dqkv[:, HQ + HK:] = d["v"]
    d["qkv"] = dqkv.view(B, T, -1)
    d["h1"], d["w_qkv"], d["b_qkv"], _ = dense.linear_backward(d["qkv"], s["h1"], w["qkv"])
    d["n1"], d["sc1"], d["sh1"] = norm.layer_norm_backward(d["h1"], s["x"], s["m1"], s["r1"], sc1, offset=1.0)
    d["x"] = d["x1"] + d["n1"]
    return d


def setting(seed):
    """Inputs; the modulation row comes from a 4-bit linear of the time embedding, the sequences' lengths differ."""
    codes = torch.randint(0, 256, (6 * C, 64), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8).to(DEV)
    weight = w4.pack(codes, (0.002 * torch.ones(6 * C, 1, device=DEV)).bfloat16(), group=128)
    mod = w4.linear(rand(B, 128, seed=seed + 20), weight)
    starts = torch.tensor([0, 70, 71, B * T - 9], dtype=torch.int32, device=DEV)      # the last 9 rows: padding
    pos = torch.arange(B * T, device=DEV)
    return dict(x=rand(B, T, C, seed=seed + 21, std=2.0), mod=mod, w=weights(seed), pos=pos,
                freq=rotary.frequencies(D).to(DEV), starts=starts), rand(B, T, C, seed=seed + 22, std=0.5)


def linear_want(x, w, b, act=None, gate=None, res=None):
    x64, w64 = x.double().flatten(0, -2), w.double()
    z, mag = torch.mm(x64, w64.t()), torch.mm(x64.abs(), w64.abs().t())
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    lead = x.shape[:-1]
    z, err = z.view(*lead, -1), ((w.shape[1] + 4) * on_dense.U * mag).view(*lead, -1)
    a = on_dense.act64(z, act)
    g = 1.0 if gate is None else gate.double()[:, None]
    y = a * g + (0.0 if res is None else res.double())
    return y, (1.13 * err + (2e-5 * a.abs() if act else 0.0)) * (g if gate is None else g.abs()) + 4 * on_dense.U * (y.abs() + (a * g).abs())


def test_forward_step_by_step():
    given, _ = setting(0)
    s, w = forward(**given), given["w"]
    sh1, sc1, g1, sh2, sc2, g2 = given["mod"].chunk(6, -1)
    on_norm.check(s["h1"], *on_norm.forward_want(s["x"], sc1, sh1, EPS, 1.0), "norm 1")
    on_dense.check(s["qkv"], *linear_want(s["h1"], w["qkv"], w["b_qkv"]), "qkv")
    spans = [(0, 70, 0, 70), (70, 71, 70, 71), (71, B * T - 9, 71, B * T - 9)]
    attn_plain.check_all(s["q"], s["k"], s["v"], spans, D ** -0.5, True, s["o"], s["lse"], what="block")
    assert (s["o"][B * T - 9:] == 0).all()
    on_dense.check(s["x1"], *linear_want(s["o"].view(B, T, -1), w["out"], None, gate=g1, res=s["x"]), "out projection")
    on_norm.check(s["h2"], *on_norm.forward_want(s["x1"], sc2, sh2, EPS, 1.0), "norm 2")
    on_dense.check(s["a"], *linear_want(s["h2"], w["up"], w["b_up"], act="gelu_tanh"), "up")
    on_dense.check(s["y"], *linear_want(s["a"], w["down"], w["b_down"], gate=g2, res=s["x1"]), "down")


def test_backward_step_by_step():
    given, dy = setting(1)
    s = forward(**given)
    d = backward(dy, s, **{k: v for k, v in given.items() if k != "x"})
    sc2 = given["mod"].chunk(6, -1)[4]
    spans = [(0, 70, 0, 70), (70, 71, 70, 71), (71, B * T - 9, 71, B * T - 9)]
    attn_plain.check_all(s["q"], s["k"], s["v"], spans, D ** -0.5, True, s["o"], None, d["o"].view(B * T, HQ, D),
                         [d["q"], d["k"], d["v"]], "block")
    assert all((d[n][B * T - 9:] == 0).all() for n in "qkv")
    want, allow, per, per_err = on_norm.backward_want(d["h2"], s["x1"], sc2, EPS, 1.0)
    on_norm.check(d["n2"], want, allow, "norm 2")
    on_norm.check(d["sc2"], per.sum(1), (per_err + 60 * on_norm.U * per.abs()).sum(1), "scale 2")
    # dx of the MLP's second half: dz = gate dy, rounded, times w.
    g = given["mod"].chunk(6, -1)[5].double()[:, None]
    dz = (dy.double() * g).flatten(0, 1)
    w64 = given["w"]["down"].double()
    h = on_dense.half(BF)
    on_dense.check(d["a"], torch.mm(dz, w64).view(B, T, F), torch.mm((h + (C + 16) * on_dense.U) * dz.abs(), w64.abs()).view(B, T, F), "da")
    assert all(torch.isfinite(v.float()).all() for v in d.values())


def test_inside_autograd():
    """The same bits through autograd, once more, and with another graph of the same leaves alive."""
    given, _ = setting(2)
    s = forward(**given)
    q, k, v = (s[n].detach().clone().requires_grad_() for n in "qkv")
    g = rand(B * T, HQ, D, seed=9)
    o = Attend.apply(q, k, v, given["starts"])
    again = Attend.apply(q, k, v, given["starts"])
    o.backward(g)
    want = attention.attention_backward(g, s["q"], s["k"], s["v"], s["o"], s["lse"], causal=True, q_starts=given["starts"])
    assert torch.equal(o, s["o"]) and torch.equal(again, o)
    assert all(torch.equal(t.grad, w) for t, w in zip((q, k, v), want))


def test_captured_and_on_another_stream():
    given, dy = setting(3)
    rest = {k: v for k, v in given.items() if k != "x"}

    def step():
        s = forward(**given)
        d = backward(dy, s, **rest)
        return [s["y"], *(v for k, v in d.items() if k != "dy")]

    want = step()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    given["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_two_streams_at_once():
    """Calls in flight together, each with its own workspaces."""
    a, b = setting(4)[0], setting(5)[0]
    want = forward(**a)["y"].clone(), forward(**b)["y"].clone()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, given in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(forward(**given)["y"])
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i % 2]) for i, t in enumerate(got))
