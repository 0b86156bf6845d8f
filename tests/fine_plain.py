"""The checkpoint with two exponents per block, in NumPy from its definition, for the
tests: no code in common with the kernels."""
import numpy as np

import train_plain as plain


def select(x):
    """1 at the two largest magnitudes of every four channels, the lower index first."""
    m, k = x.shape
    order = np.argsort(-np.abs(x).reshape(m, -1, 4), axis=-1, kind="stable")
    mk = np.zeros((m, k // 4, 4))
    np.put_along_axis(mk, order[..., :2], 1.0, -1)
    return mk.reshape(m, k)


def pack_fine(x, mk):
    """(codes, exps, pruned_exps) of fp64 x [m, k] that holds bf16 values."""
    kept, exps = plain.pack(x * mk)
    codes, pruned = plain.pack(x * (1 - mk))
    codes = np.where((codes == 0) & (x != 0), np.sign(x), codes)   # no nonzero pruned channel has code 0
    return np.where(mk == 1, kept, codes).astype(np.int8), exps, pruned


def values_fine(codes, exps, pruned, mk):
    return np.where(mk == 1, plain.values(codes, exps), plain.values(codes, pruned))
