"""The rest of a transformer block next to the sparse layer, as it is measured.

Layer norm with a weight and bias per channel or per sequence, the dense linear
layer with bias, activation, gate and residual in its epilogue, and attention
(whole sequences, packed sequences, a cache), each forward and, for training,
forward and backward.  Each in a plain form of elementary torch operations, as
the framework's own call, and as a 64-bit evaluation of its definition.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one new token's norm before a projection: latency
        dict(name="norm_one_token", op="norm", back=False, dtype="bfloat16", b=1, t=1, c=4096, affine="shared", offset=0.0),
        # 2 x (4096 image + 512 text) tokens, scale and shift of each image from its modulation row
        dict(name="norm_modulated", op="norm", back=False, dtype="bfloat16", b=2, t=4608, c=4096, affine="sequence",
             offset=1.0),
        # a training step of a ragged batch, odd channel count
        dict(name="norm_train_ragged", op="norm", back=True, dtype="float16", b=3, t=1155, c=1028, affine="sequence",
             offset=1.0),
        # a training step of an ordinary norm over many tokens
        dict(name="norm_train", op="norm", back=True, dtype="bfloat16", b=4, t=2048, c=4096, affine="shared", offset=0.0),
        # a few rows: pooled text into a hidden layer, an odd number of outputs
        dict(name="linear_few_rows", op="linear", back=False, dtype="bfloat16", m=3, k=4096, n=4099, act="silu", bias=True,
             gate="none", residual=False, b=1),
        # the MLP's first half of one image
        dict(name="linear_mlp_up", op="linear", back=False, dtype="bfloat16", m=4096, k=4096, n=12288, act="gelu_tanh",
             bias=True, gate="none", residual=False, b=1),
        # an output projection into the residual stream, one gate row per sequence, ragged
        dict(name="linear_gate_residual", op="linear", back=False, dtype="float16", m=2310, k=1152, n=1160, act="none",
             bias=True, gate="sequence", residual=True, b=2),
        # a training step of an MLP's first half
        dict(name="linear_train", op="linear", back=True, dtype="bfloat16", m=4096, k=2048, n=8192, act="gelu", bias=True,
             gate="none", residual=False, b=1),
        # one new token each of eight sequences over a long cache, query heads sharing key heads
        dict(name="attn_one_token", op="attn", form="cache", back=False, causal=True, dtype="bfloat16", b=8, tq=1,
             tk=16384, hq=32, hk=8, d=128, mix=1),
        # a block's attention over 2 x (4096 image + 512 text) tokens
        dict(name="attn_image_text", op="attn", form="batch", back=False, causal=False, dtype="bfloat16", b=2, tq=4608,
             tk=4608, hq=24, hk=24, d=128, mix=2),
        # prompts of different lengths in one row of tokens, text encoder heads
        dict(name="attn_packed", op="attn", form="packed", back=False, causal=True, dtype="float16", b=9, tq=1000, tk=1000,
             hq=20, hk=4, d=72, mix=3),
        # a training step's attention over one packed batch
        dict(name="attn_train", op="attn", form="packed", back=True, causal=False, dtype="bfloat16", b=4, tq=1800, tk=1800,
             hq=16, hk=8, d=128, mix=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "attn"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op == "norm":
        c = _log_int(rng, 24, 12000) if rng.random() < 0.4 else 8 * _log_int(rng, 4, 1500)
        b = rng.randint(1, 4)
        return dict(op="norm", back=rng.random() < 0.5, dtype=rng.choice([dtype, "float32"]), b=b,
                    t=_log_int(rng, 1, min(8000, 30_000_000 // (b * c))), c=c,
                    affine=rng.choice(["none", "shared", "sequence"]), offset=rng.choice([0.0, 1.0]))
    if op == "linear":
        b, back = rng.randint(1, 3), rng.random() < 0.4
        m, k = b * _log_int(rng, 1, 1300), 8 * _log_int(rng, 8, 512)
        most = 400_000_000_000 // (m * k * (6 if back else 2))     # no costlier than the listed ones
        return dict(op="linear", back=back, dtype=dtype, m=m, k=k, n=_log_int(rng, 24, min(9000, most)), act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.7, gate=rng.choice(["none", "none", "shared", "sequence"]),
                    residual=rng.random() < 0.5, b=b)
    form = rng.choice(["batch", "packed", "cache"])
    hk = rng.randint(1, 6)
    d = rng.choice([32, 40, 64, 72, 96, 128])
    group = rng.randint(1, 4)
    causal = rng.random() < 0.5
    mix = rng.randrange(1 << 20)
    if form == "cache":
        return dict(op="attn", form=form, back=False, causal=True, dtype=dtype, b=rng.randint(1, 8), tq=_log_int(rng, 1, 24),
                    tk=_log_int(rng, 40, 30_000), hq=hk * group, hk=hk, d=d, mix=mix)
    b, back = rng.randint(1, 6), rng.random() < 0.5
    most = 450_000_000_000 / (b * hk * group * d * (14 if back else 4) * (4 if form == "packed" else 1))
    most = min(3000, int(math.sqrt(most)))                         # no costlier than the listed ones
    tq = _log_int(rng, 1, most)
    tk = tq if form == "packed" or rng.random() < 0.5 else _log_int(rng, 1, most)
    return dict(op="attn", form=form, back=back, causal=causal, dtype="bfloat16" if back else dtype, b=b, tq=tq, tk=tk,
                hq=hk * group, hk=hk, d=d, mix=mix)


def _lengths(case):
    """Packed: tokens of each sequence.  Cache: filled rows of each sequence."""
    r = random.Random(case["mix"])
    if case["form"] == "packed":
        return [r.randint(1, 2 * case["tq"] - 1) for _ in range(case["b"])]
    if case["form"] == "cache":
        return [r.randint((case["tk"] + 1) // 2, case["tk"]) for _ in range(case["b"])]
    return [case["tk"]] * case["b"]


def _pairs(case):
    """Query-key pairs of one head."""
    total = 0
    for n in _lengths(case):
        tq = n if case["form"] == "packed" else case["tq"]
        if not case["causal"]:
            total += tq * n
        else:                                                      # query i sees keys up to i + n - tq
            first = max(0, tq - n)
            rows = tq - first
            total += rows * (first + n - tq + 1) + rows * (rows - 1) // 2
    return total


def work(case):
    c = case
    if c["op"] == "norm":
        n, size = c["b"] * c["t"] * c["c"], 4 if c["dtype"] == "float32" else 2
        rows = {"none": 0, "shared": 1, "sequence": c["b"]}[c["affine"]]
        extra = 2 * rows * c["c"] * size
        if not c["back"]:
            return {"bytes": 2 * n * size + extra, "flops": 8 * n}
        return {"bytes": 5 * n * size + 2 * extra, "flops": 20 * n}
    if c["op"] == "linear":
        m, k, n = c["m"], c["k"], c["n"]
        bytes_ = 2 * (m * k + n * k + m * n * (2 if c["residual"] else 1))
        if not c["back"]:
            return {"bytes": bytes_, "flops": 2 * m * n * k}
        return {"bytes": bytes_ + 2 * (2 * m * n + 2 * m * k + 2 * n * k), "flops": 6 * m * n * k}
    lens = _lengths(c)
    tq = sum(lens) if c["form"] == "packed" else c["b"] * c["tq"]
    rows = tq * c["hq"] + sum(lens) * c["hk"]                      # of q and o, of k and v
    f = 4 * _pairs(c) * c["hq"] * c["d"]
    if not c["back"]:
        return {"bytes": 4 * rows * c["d"], "flops": f}
    return {"bytes": 4 * rows * c["d"] + 2 * (4 * tq * c["hq"] + 4 * sum(lens) * c["hk"]) * c["d"], "flops": f * 7 // 2}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    dtype = getattr(torch, c["dtype"])

    def normal(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device=DEV)).to(dtype)

    st = dict(case=c)
    if c["op"] == "norm":
        b, t, n = c["b"], c["t"], c["c"]
        x = torch.randn(b, t, n, generator=g, device=DEV)
        hot = torch.rand(n, generator=g, device=DEV) < 0.02       # a few channels far from the rest, as in a residual stream
        st["x"] = (torch.where(hot, 12.0 * x + 6.0, x) + 0.3).to(dtype)
        st["weight"] = st["bias"] = None
        if c["affine"] == "sequence":                              # slices of a modulation row of six vectors
            rows = normal(b, 6 * n, std=0.2)
            st["weight"], st["bias"] = rows[:, n:2 * n], rows[:, :n]
        elif c["affine"] == "shared":
            st["weight"] = (normal(n, std=0.2).float() + 1.0 - c["offset"]).to(dtype)
            st["bias"] = normal(n, std=0.2)
        if c["back"]:
            st["dy"] = normal(b, t, n, std=0.5)
        return st
    if c["op"] == "linear":
        m, k, n, b = c["m"], c["k"], c["n"], c["b"]
        st["x"] = normal(b, m // b, k)
        st["w"] = normal(n, k, std=k ** -0.5)
        st["bias"] = normal(n, std=0.2) if c["bias"] else None
        st["gate"] = None if c["gate"] == "none" else normal(n) if c["gate"] == "shared" else normal(b, 6 * n)[:, 2 * n:3 * n]
        st["residual"] = normal(b, m // b, n, std=2.0) if c["residual"] else None
        if c["back"]:
            st["dy"] = normal(b, m // b, n, std=0.5)
        return st
    b, hq, hk, d = c["b"], c["hq"], c["hk"], c["d"]
    lens = _lengths(c)
    st["starts"] = st["k_lens"] = None
    if c["form"] == "packed":                                      # slices of one projection's output
        total = sum(lens)
        qkv = normal(total, hq + 2 * hk, d)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        st["starts"] = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32, device=DEV)
        st["most"] = max(lens)                                     # the plain form's padding
    else:
        st["q"] = normal(b, c["tq"], hq, d)
        st["k"], st["v"] = normal(b, c["tk"], hk, d), normal(b, c["tk"], hk, d)
        if c["form"] == "cache":
            st["k_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if c["back"]:
        st["do"] = normal(*st["q"].shape, std=0.5)
    return st


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _act(z, name):
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, name):
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _rows(v):
    """A vector per channel or per sequence, to broadcast over [batch, tokens, channels]."""
    return v.float()[:, None] if v.dim() == 2 else v.float()


def _norm(st):
    c = st["case"]
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5)
    xhat = (x - mean) * rstd
    dtype = st["x"].dtype
    factor = 1.0 if st["weight"] is None else _rows(st["weight"]) + c["offset"]
    y = xhat * factor
    if st["bias"] is not None:
        y = y + _rows(st["bias"])
    if not c["back"]:
        return y.to(dtype)
    dy = st["dy"].float()
    g = dy * factor
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    if st["weight"] is None:
        return y.to(dtype), dx.to(dtype)
    over = (1,) if c["affine"] == "sequence" else (0, 1)
    return y.to(dtype), dx.to(dtype), (dy * xhat).sum(over).to(dtype), dy.sum(over).to(dtype)


def _linear(st):
    c = st["case"]
    dtype = st["x"].dtype
    x, w = st["x"].float(), st["w"].float()
    z = x @ w.t()
    if st["bias"] is not None:
        z = z + st["bias"].float()
    a = _act(z, c["act"])
    y = a if st["gate"] is None else a * _rows(st["gate"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    if not c["back"]:
        return y.to(dtype)
    dy = st["dy"].float()
    dz = dy * _act_slope(z, c["act"])
    if st["gate"] is not None:
        dz = dz * _rows(st["gate"])
    flat = dz.flatten(0, 1)
    outs = [y.to(dtype), (dz @ w).to(dtype), (flat.t() @ x.flatten(0, 1)).to(dtype)]
    if st["bias"] is not None:
        outs.append(flat.sum(0).to(dtype))
    if st["gate"] is not None:
        outs.append((dy * a).sum((1,) if c["gate"] == "sequence" else (0, 1)).to(dtype))
    return tuple(outs)


def _padded(x, at):
    """Rows of a packed tensor [n, heads, d] at the indices [sequences, most], heads first, in fp32."""
    return x.float()[at].transpose(1, 2)


def _attention(st):
    c = st["case"]
    hq, hk, d, causal = c["hq"], c["hk"], c["d"], c["causal"]
    group, dtype = hq // hk, st["q"].dtype
    packed = c["form"] == "packed"
    if packed:
        starts = st["starts"].long()
        len_q = len_k = starts[1:] - starts[:-1]
        at = torch.arange(st["most"], device=DEV)
        at = torch.minimum(starts[:-1, None] + at, starts[1:, None] - 1)
        q, k, v = (_padded(st[n], at) for n in "qkv")
    else:
        q, k, v = (st[n].float().transpose(1, 2) for n in "qkv")
        b = c["b"]
        len_q = torch.full((b,), c["tq"], device=DEV)
        len_k = len_q.new_full((b,), c["tk"]) if st["k_lens"] is None else st["k_lens"].long()
    b, tq, tk = q.shape[0], q.shape[2], k.shape[2]
    i, j = torch.arange(tq, device=DEV), torch.arange(tk, device=DEV)
    seen = (j < len_k[:, None])[:, None, :] & (i < len_q[:, None])[:, :, None]
    if causal:
        seen = seen & (j <= i[:, None] + (len_k - len_q)[:, None, None])
    seen = seen[:, None, None]                                     # [b, 1, 1, tq, tk]
    q = q.reshape(b, hk, group * tq, d)
    k, v = k.contiguous(), v.contiguous()
    scale = d ** -0.5
    s = (q @ k.transpose(2, 3).contiguous()).view(b, hk, group, tq, tk) * scale
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    p = p.view(b, hk, group * tq, tk)
    o = p @ v                                                      # [b, hk, group * tq, d]
    if packed:
        seq = torch.repeat_interleave(torch.arange(b, device=DEV), len_q, output_size=st["q"].shape[0])
        row = torch.arange(st["q"].shape[0], device=DEV) - starts[seq]

    def back(t, heads):
        t = t.view(b, heads, -1, d).transpose(1, 2)
        return (t[seq, row] if packed else t).to(dtype).contiguous()

    if not c["back"]:
        return back(o, hq)
    do = _padded(st["do"], at) if packed else st["do"].float().transpose(1, 2)
    if packed:                                                     # the padding's rows have no gradient
        do = do * (i < len_q[:, None])[:, None, :, None]
    do = do.reshape(b, hk, group * tq, d)
    ds = p * (do @ v.transpose(2, 3).contiguous() - (do * o).sum(-1, keepdim=True)) * scale
    return (back(o, hq), back(ds @ k, hq), back(ds.transpose(2, 3).contiguous() @ q, hk),
            back(p.transpose(2, 3).contiguous() @ do, hk))


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"norm": _norm, "linear": _linear, "attn": _attention}[c["op"]](state)
    st = state
    if c["op"] == "norm":
        from activation_sparse_gemm_token_amd import norm
        if not c["back"]:
            return norm.layer_norm(st["x"], st["weight"], st["bias"], offset=c["offset"])
        y, mean, rstd = norm.layer_norm(st["x"], st["weight"], st["bias"], offset=c["offset"], return_stats=True)
        dx, dw, db = norm.layer_norm_backward(st["dy"], st["x"], mean, rstd, st["weight"], offset=c["offset"])
        return (y, dx) if dw is None else (y, dx, dw, db)
    if c["op"] == "linear":
        from activation_sparse_gemm_token_amd import dense
        act = None if c["act"] == "none" else c["act"]
        if not c["back"]:
            return dense.linear(st["x"], st["w"], st["bias"], activation=act, gate=st["gate"], residual=st["residual"])
        y, z = dense.linear(st["x"], st["w"], st["bias"], activation=act, gate=st["gate"], residual=st["residual"],
                            keep=True)
        grads = dense.linear_backward(st["dy"], st["x"], st["w"], z, activation=act, gate=st["gate"],
                                      need_dbias=st["bias"] is not None)
        return (y, *(t for t in grads if t is not None))
    from activation_sparse_gemm_token_amd import attention
    if not c["back"]:
        return attention.attention(st["q"], st["k"], st["v"], causal=c["causal"], q_starts=st["starts"], k_lens=st["k_lens"])
    o, lse = attention.attention(st["q"], st["k"], st["v"], causal=c["causal"], q_starts=st["starts"], k_lens=st["k_lens"],
                                 return_lse=True)
    return (o, *attention.attention_backward(st["do"], st["q"], st["k"], st["v"], o, lse, causal=c["causal"],
                                             q_starts=st["starts"], k_lens=st["k_lens"]))


# --------------------------------------------------------------------------
# The definitions in 64 bits: the forward pass, and its gradients by differentiation
# --------------------------------------------------------------------------

def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _gradients(y, leaves, dy):
    leaves = [t for t in leaves if t is not None]
    return (y.detach(), *torch.autograd.grad(y, leaves, dy.double()))


def _per_row(v, b, t, n):
    """[n] or [b, n] as one row for each of b * t tokens."""
    return (v.expand(b, n) if v.dim() == 1 else v).repeat_interleave(t, 0)


def _exact_norm(st):
    c = st["case"]
    b, t, n = c["b"], c["t"], c["c"]
    x, w, bias = _leaf(st["x"]), _leaf(st["weight"]), _leaf(st["bias"])
    v = x.reshape(b * t, n)
    var, mean = torch.var_mean(v, 1, correction=0, keepdim=True)
    y = (v - mean) * torch.rsqrt(var + 1e-5)
    if w is not None:
        y = y * (_per_row(w, b, t, n) + c["offset"]) + _per_row(bias, b, t, n)
    y = y.view(b, t, n)
    return _gradients(y, (x, w, bias), st["dy"]) if c["back"] else y.detach()


def _exact_linear(st):
    c = st["case"]
    b, m, n = c["b"], c["m"], c["n"]
    x, w, bias, gate = (_leaf(st[k]) for k in ("x", "w", "bias", "gate"))
    z = torch.mm(x.reshape(m, -1), w.t())
    if bias is not None:
        z = z + bias[None]
    half = math.sqrt(2.0 / math.pi)
    if c["act"] == "gelu":
        z = z * (1.0 - 0.5 * torch.erfc(z / math.sqrt(2.0)))
    elif c["act"] == "gelu_tanh":                                  # (1 + tanh u) / 2 is 1 / (1 + e^-2u)
        z = z * torch.sigmoid(2.0 * half * (z + 0.044715 * z.pow(3)))
    elif c["act"] == "silu":
        z = z * torch.sigmoid(z)
    if gate is not None:
        z = z * _per_row(gate, b, m // b, n)
    if st["residual"] is not None:
        z = z + st["residual"].double().view(m, n)
    y = z.view(b, m // b, n)
    return _gradients(y, (x, w, bias, gate), st["dy"]) if c["back"] else y.detach()


def _exact_attn(st):
    c = st["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    lens = _lengths(c)
    packed = c["form"] == "packed"
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    grads = [torch.zeros(st[n].shape, dtype=torch.float64, device=DEV) for n in "qkv"]
    first = 0
    for b, n in enumerate(lens):
        qs = (slice(first, first + n),) if packed else (b, slice(None))
        ks = qs if packed else (b, slice(0, n))
        first += n
        for h in range(hq):
            iq, ik = (*qs, h), (*ks, h // (hq // hk))
            q, k, v = (st[m][i].double().requires_grad_(c["back"]) for m, i in (("q", iq), ("k", ik), ("v", ik)))
            s = torch.mm(q, k.t()) / math.sqrt(d)
            if c["causal"]:
                hidden = torch.ones_like(s, dtype=torch.bool).triu(1 + s.shape[1] - s.shape[0])
                s = s.masked_fill(hidden, -math.inf)
            p = torch.softmax(s, 1)
            if c["causal"] and s.shape[0] > s.shape[1]:            # the first queries see nothing
                p = torch.where(hidden.all(1, keepdim=True), 0.0, p)
            y = torch.mm(p, v)
            o[iq] = y.detach()
            if c["back"]:
                for t, i, dt in zip(grads, (iq, ik, ik), torch.autograd.grad(y, (q, k, v), st["do"][iq].double())):
                    t[i] += dt
    return (o, *grads) if c["back"] else o


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "attn": _exact_attn}[case["op"]](st)
