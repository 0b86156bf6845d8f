"""Every form of the layer's backward pass, all of dX, dA and dB against fp64 on the
device: tiles of G W (256, 192 and 64 columns, one contraction range and several,
padded rows, channel tails) and the main loops of the LoRA products (three steps of
a wavefront and more).  Each case asserts the form that it is here for.

Tolerances: half a bf16 step of the result, and what fp32 sums lose: depth() roundings
of 2^-24 of the magnitudes summed, through every later product (train_plain.depth)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from activation_sparse_gemm_token_amd import training  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_plain as plain  # noqa: E402

DEV = "cuda:0"
U24, HALF, depth = plain.U24, plain.HALF_BF16, plain.depth


def say(*a):
    print("[forms]", *a, file=sys.stderr, flush=True)


def make(m, n, k, r):
    g = torch.Generator(device=DEV).manual_seed(m + n + k + r)
    rand = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device=DEV)).bfloat16()  # noqa: E731
    hot = torch.rand(m, k, generator=g, device=DEV) < 0.08         # a few large channels, the rest small
    x = torch.where(hot, 4.0, 0.3).bfloat16() * rand(m, k)
    return dict(kept=training.checkpoint(x), g=rand(m, n, std=0.01), w_t=rand(k, n, std=0.02), a=rand(r, k, std=0.05),
                b=rand(n, r, std=0.05))


def mask(idx, k):
    code = torch.stack([idx & 15, idx >> 4], -1).flatten(1)[:, :k // 4].int()
    at = torch.arange(4, device=DEV)
    return ((at == (code & 3)[..., None]) | (at == (code >> 2)[..., None])).flatten(1).double()


def t(v):
    return v.t().contiguous()


def reference(d, alpha):
    """((dx, da, db), tolerances)."""
    kept = d["kept"]
    m, k = kept.m, kept.k
    g, w, a, b = (d[i].double() for i in ("g", "w_t", "a", "b"))
    n, r = b.shape
    x, mk = kept.unpack().double(), mask(kept.idx, k)
    s, lk = kept.stats[:, :1].double(), kept.stats[:, 1:].double()
    inv = torch.where(lk > 0, 1 / lk, 0.0)
    G, A, B, X, al = g.abs(), a.abs(), b.abs(), x.abs(), abs(alpha)
    u = alpha * (g @ b)
    du = depth(n) * U24 * al * (G @ B)
    U = u.abs()
    v = u @ a
    dv = du @ A + (3 * r + 4) * U24 * (U @ A)                      # three words each
    p = g @ t(w)
    dp = depth(n) * U24 * (G @ t(w.abs()))
    e = p - v
    ka = (mk * x) @ t(a)
    dka = depth(k) * U24 * ((mk * X) @ t(A))
    D = (mk * x * e).sum(1, keepdim=True)
    dD = (mk * X * (dp + depth(k) * U24 * p.abs())).sum(1, keepdim=True) + \
        (du * ka.abs() + U * dka + (r + 4) * U24 * U * ka.abs()).sum(1, keepdim=True)
    turn = torch.sign(x) * (1 - s * mk)
    dx = v + s * mk * e + D * inv * turn
    tol_x = HALF * dx.abs() + (1 - s * mk).abs() * dv + s * mk * dp + dD * inv * turn.abs() + \
        8 * U24 * (v.abs() * (1 + s) + s * p.abs() + (D * inv).abs())
    rest = x * (1 - s * mk)
    R = rest.abs()
    da = t(u) @ rest
    tol_a = HALF * da.abs() + t(du + 4 * U24 * U) @ R + 3 * depth(m) * U24 * (t(U) @ R)
    tt = alpha * (rest @ t(a))
    db = t(g) @ tt
    tol_b = HALF * db.abs() + t(G) @ (al * depth(k) * U24 * (R @ t(A))) + 3 * depth(m) * U24 * (t(G) @ tt.abs())
    return (dx, da, db), (tol_x, tol_a, tol_b)


def check(m, n, k, r, alpha=0.5):
    d = make(m, n, k, r)
    ws = torch.full((training.backward_workspace_bytes(m, n, k, r),), 0xff, dtype=torch.uint8, device=DEV)
    got = training.sparse_linear_backward(d["g"], d["kept"], d["w_t"], d["a"], d["b"], alpha, workspace=ws)
    want, tol = reference(d, alpha)
    off = {name: int((~((y.double() - w).abs() <= e)).sum()) for name, y, w, e in zip(("dx", "da", "db"), got, want, tol)}
    assert off == {"dx": 0, "da": 0, "db": 0}


# (m, n, k), tile columns, several ranges, padded rows
TILES = [((65, 32, 128), 64, False, False), ((66, 32, 140), 64, False, False), ((69, 572, 136), 64, True, False),
         ((71, 512, 148), 64, True, False), ((77, 1580, 9152), 64, True, False),
         ((414, 32, 7304), 192, False, False), ((3459, 32, 860), 192, False, False), ((4519, 64, 696), 192, False, False),
         ((4939, 64, 604), 192, False, False), ((4788, 36, 848), 192, False, True), ((2260, 36, 1820), 192, False, True),
         ((94, 1072, 9224), 192, True, False), ((130, 1112, 5956), 192, True, False), ((283, 1088, 3368), 192, True, False),
         ((360, 1152, 2756), 192, True, False), ((667, 564, 2984), 192, True, True), ((1246, 524, 1660), 192, True, True),
         ((2522, 32, 4808), 256, False, False), ((1331, 32, 8764), 256, False, False), ((1605, 64, 7368), 256, False, False),
         ((1308, 64, 9124), 256, False, False), ((1419, 36, 8264), 256, False, True), ((2600, 36, 4428), 256, False, True),
         ((588, 1352, 8712), 256, True, False), ((520, 1392, 8884), 256, True, False), ((573, 1408, 8536), 256, True, False),
         ((592, 2048, 8236), 256, True, False), ((792, 1356, 6488), 256, True, True), ((614, 1580, 8092), 256, True, True)]


@pytest.mark.parametrize("size,columns,ranges,padded", TILES)
def test_tiles(size, columns, ranges, padded):
    m, n, k = size
    say(m, n, k)
    form = training.backward_form(m, n, k, 16)
    assert form[0] == columns and (form[1] > 1) == ranges and form[2] == (n + 4 if padded else n)
    check(m, n, k, 16)


# (m, n, k, r), the least steps of a wavefront over G's channels, the checkpoint's, and the tokens
LOOPS = [((1300, 6404, 3108, 48), (3, 3, 3)), ((1300, 6400, 3112, 64), (3, 3, 3)), ((2050, 6404, 3108, 64), (4, 5, 4)),
         ((2050, 6400, 3112, 33), (4, 5, 4)), ((2050, 6404, 3112, 100), (9, 13, 5)), ((2050, 6400, 3108, 128), (9, 13, 5)),
         ((2100, 6404, 3112, 16), (4, 5, 4)), ((2100, 6400, 3108, 32), (4, 5, 4)), ((4100, 520, 6152, 128), (3, 20, 7)),
         ((6100, 4612, 260, 65), (18, 2, 5))]


@pytest.mark.parametrize("size,least", LOOPS)
def test_main_loops(size, least):
    say(*size)
    form = training.backward_form(*size)
    steps = (form[3] // 256, form[4] // 256, form[5] // 128)
    assert all(s >= want for s, want in zip(steps, least)), steps
    check(*size)
