"""Attention of one sequence and head in fp64, with what the kernels' roundings allow.

U is fp32's half step, H the tensors' type's.  A weight p is off by its own rounding (H), by
its score's error (a sum of d products, scaled) and by the exponential's few steps; a sum of n
terms by n U of the terms' magnitudes; a result by H of itself.  fp16 weights below its normal
range are off by 2^-25 of the largest one instead."""
import math

import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def visible(nq, nk, causal, dev):
    m = torch.ones(nq, nk, dtype=torch.bool, device=dev)
    return m.tril(nk - nq) if causal else m


def one(q, k, v, scale, causal, d_o=None, few=False):
    """q [nq, d], k, v [nk, d] of one head: dict of o, lse and (with d_o) dq, dk, dv, each a pair
    (value, allowance), fp64.  ``few``: D is formed from p and dP, not from the rounded o (up to 128 keys)."""
    h, dtype = half(q.dtype), q.dtype
    q, k, v = (t.double() for t in (q, k, v))
    (nq, d), nk = q.shape, k.shape[0]
    seen = visible(nq, nk, causal, q.device)
    raw = torch.mm(q, k.t())
    s = torch.where(seen, raw * scale, -math.inf)
    if nk:
        top = s.amax(1, keepdim=True)
        top = torch.where(torch.isinf(top), 0.0, top)
    else:
        top = torch.zeros(nq, 1, dtype=torch.float64, device=q.device)
    e = torch.exp(s - top)
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / torch.where(total > 0, total, 1.0), 0.0)
    o = torch.mm(p, v)
    lse = torch.where(total > 0, torch.log(torch.where(total > 0, total, 1.0)) + top, -math.inf)[:, 0]
    # Error of a score (then relative error of a weight): products, the scaling, the subtraction.
    ds_ = (d + 4) * U * scale * torch.mm(q.abs(), k.abs().t()) + 8 * U * (s.abs().nan_to_num(posinf=0) + top.abs())
    ds_ = torch.where(seen, ds_, 0.0)
    most = ds_.amax(1, keepdim=True) if nk else torch.zeros_like(top)
    rel = h + ds_ + most + (2 * nk + 32) * U
    tiny = 2.0 ** -25 if dtype is torch.float16 else 0.0
    pe = torch.where(seen, p * rel + tiny / torch.where(total > 0, total, 1.0), 0.0)
    out = {"o": (o, h * o.abs() + torch.mm(pe, v.abs()) + 2.0 ** -25 * (dtype is torch.float16)),
           "lse": (lse, most[:, 0] + (2 * nk + 32) * U + 4 * U * lse.abs().nan_to_num(posinf=0))}
    if d_o is None:
        return out
    g = d_o.double()
    dp = torch.mm(g, v.t())
    dd = (g * o).sum(1, keepdim=True)
    ds = p * (dp - dd)
    # D is formed from the rounded o, dP from d products.
    o_err = out["o"][1]
    dd_err = (g.abs() * o_err).sum(1, keepdim=True) + (d + 4) * U * (g.abs() * o.abs()).sum(1, keepdim=True)
    dp_err = (d + 4) * U * torch.mm(g.abs(), v.abs().t())
    p_err = p * (ds_ + most + (2 * nk + 48) * U)
    if few:
        dd_err = (p_err * dp.abs() + p * dp_err + (nk + 8) * U * p * dp.abs()).sum(1, keepdim=True)
    ds_err = h * ds.abs() + (1 + h) * (p_err * (dp - dd).abs() + (p + p_err) * (dp_err + dd_err + 4 * U * (dp.abs() + dd.abs())))
    n = 2 * (nq + nk) * U
    out["dv"] = (torch.mm(p.t(), g), torch.mm((p_err + h * p + n * p).t(), g.abs()))
    out["dk"] = (scale * torch.mm(ds.t(), q), scale * torch.mm((ds_err + n * ds.abs()).t(), q.abs()))
    out["dq"] = (scale * torch.mm(ds, k), scale * torch.mm(ds_err + n * ds.abs(), k.abs()))
    return out


def check(got, want, allow, what):
    """|got - want| <= allow, with the result's own rounding added."""
    g = got.double()
    a = allow + half(got.dtype) * want.abs() * 1.01 if got.dtype is not torch.float32 else allow
    same = torch.isinf(want) & (g == want)
    bad = ~(((g - want).abs() <= a) | same)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(g[tuple(i)])} for "
                             f"{float(want[tuple(i)])}, allowed {float(a[tuple(i)]):.3g}")


def check_all(q, k, v, spans, scale, causal, o, lse=None, d_o=None, grads=None, what=""):
    """Packed [tokens, heads, d] tensors and spans [(q0, q1, k0, k1)]; lse [heads, tokens].  Checks the
    rows of the spans."""
    hq, hk = q.shape[1], k.shape[1]
    g = hq // hk
    for n, (q0, q1, k0, k1) in enumerate(spans):
        for j in range(hk):
            dk = dv = dka = dva = 0
            for h in range(j * g, (j + 1) * g):
                r = one(q[q0:q1, h], k[k0:k1, j], v[k0:k1, j], scale, causal, None if d_o is None else d_o[q0:q1, h])
                w = f"{what} sequence {n} head {h}"
                check(o[q0:q1, h], *r["o"], w + " o")
                if lse is not None:
                    check(lse[h, q0:q1], *r["lse"], w + " lse")
                if grads is not None:
                    check(grads[0][q0:q1, h], *r["dq"], w + " dq")
                    dk, dka = dk + r["dk"][0], dka + r["dk"][1]
                    dv, dva = dv + r["dv"][0], dva + r["dv"][1]
            if grads is not None:
                check(grads[1][k0:k1, j], dk, dka, w + " dk")
                check(grads[2][k0:k1, j], dv, dva, w + " dv")
