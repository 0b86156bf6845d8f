"""The checkpoint and the layer's gradients in NumPy fp64, from their
definitions, for the GPU tests: no code in common with the kernels."""
import numpy as np

U24, U16, HALF_BF16 = 2.0 ** -24, 2.0 ** -16, 2.0 ** -8


def bf16(t):
    return t.detach().cpu().double().numpy()


def pack(x):
    """(codes, exps) of fp64 x [m, k] that holds bf16 values."""
    m, k = x.shape
    codes, exps = np.zeros((m, k), np.int8), np.zeros((m, -(-k // 32)), np.uint8)
    for b in range(exps.shape[1]):
        blk = x[:, 32 * b:32 * b + 32]
        amax = np.abs(blk).max(1)
        e = np.full(m, -133)
        some = amax > 0
        e[some] = np.maximum(np.floor(np.log2(amax[some])).astype(int) - 6, -133)
        exps[:, b] = e + 133
        codes[:, 32 * b:32 * b + 32] = np.clip(np.rint(blk / 2.0 ** e[:, None].astype(float)), -127, 127)
    return codes, exps


def values(codes, exps):
    k = codes.shape[1]
    return codes.astype(np.float64) * np.repeat(2.0 ** (exps.astype(np.float64) - 133), 32, 1)[:, :k]


def mask(idx, k):
    code = np.stack([idx & 15, idx >> 4], -1).reshape(idx.shape[0], -1)[:, :k // 4]
    at = np.arange(4)
    return ((at == (code & 3)[..., None]) | (at == (code >> 2)[..., None])).reshape(idx.shape[0], k).astype(np.float64)


def depth(n, parts=32):
    """Roundings an element of a length-n sum can pass: 32 inside a matrix
    instruction, one per instruction, one per range joined, a few on the way."""
    return n / 32 + 40 + parts


def backward(g, x, mk, s, lk, w_t, a, b, alpha):
    """Gradients (dx, da, db) and how far the kernel's may be from them: half a
    bf16 step each, the fp32 sums of depth() roundings, and U and T carried as
    two bf16 words (2^-16 of the value)."""
    (m, n), k, r = g.shape, x.shape[1], a.shape[0]
    s, lk = s[:, None], lk[:, None]
    inv = np.where(lk > 0, 1 / np.where(lk > 0, lk, 1), 0)
    A, B, G, X = np.abs(a), np.abs(b), np.abs(g), np.abs(x)
    u = alpha * g @ b
    du = depth(n) * U24 * abs(alpha) * (G @ B)
    v = u @ a
    U = np.abs(u)
    dv = (du + U16 * U) @ A + (2 * r + 4) * U24 * (U @ A)
    p = g @ w_t.T
    dp = depth(n) * U24 * (G @ np.abs(w_t).T)
    e = p - v
    ka = (mk * x) @ a.T
    dka = depth(k) * U24 * ((mk * X) @ A.T)
    d = (mk * x * e).sum(1, keepdims=True)
    dd = (mk * X * (dp + depth(k) * U24 * np.abs(p))).sum(1, keepdims=True) + \
        (du * np.abs(ka) + U * dka + (r + 4) * U24 * U * np.abs(ka)).sum(1, keepdims=True)
    turn = np.sign(x) * (1 - s * mk)
    dx = v + s * mk * e + d * inv * turn
    tol_x = HALF_BF16 * np.abs(dx) + np.abs(1 - s * mk) * dv + s * mk * dp + dd * inv * np.abs(turn) + \
        8 * U24 * (np.abs(v) * (1 + s) + s * np.abs(p) + np.abs(d * inv))
    rest = x * (1 - s * mk)
    R = np.abs(rest)
    da = u.T @ rest
    tol_a = HALF_BF16 * np.abs(da) + (du + (U16 + 4 * U24) * U).T @ R + depth(m) * U24 * (U.T @ R)
    t = alpha * rest @ a.T
    T = np.abs(t)
    dt = abs(alpha) * depth(k) * U24 * (R @ A.T) + U16 * T
    db = g.T @ t
    tol_b = HALF_BF16 * np.abs(db) + G.T @ dt + depth(m) * U24 * (G.T @ T)
    return (dx, da, db), (tol_x, tol_a, tol_b)


def forward(x, mk, w, a, b, alpha):
    """The layer in fp64, s from x itself: what the gradients are of."""
    lk = (mk * np.abs(x)).sum(1, keepdims=True)
    s = np.where(lk > 0, np.abs(x).sum(1, keepdims=True) / np.where(lk > 0, lk, 1), 1.0)
    kept = s * mk * x
    return kept @ w.T + alpha * ((x - kept) @ a.T) @ b.T
