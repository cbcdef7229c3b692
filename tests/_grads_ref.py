"""The gradient operators' definitions in float64 NumPy, and the error bounds
their float32 arithmetic keeps, for the tests of include/ma_grads.h.

A rounding to a type errs by at most half a step, U[type] relative to the
value.  `tol` arrays are absolute bounds per element."""

import numpy as np

U = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
F32 = 2.0 ** -24
UNDER = 2.0 ** -126    # the smallest normal float32
TINY = 1e-37       # results that underflow


def pitches(cols):
    cp = -(-cols // 32) * 32
    return cp, -(-cp // 128) * 4


def pack(x):
    """(codes, exps) of float64 x (holding float32 or bf16 values): the
    definition in include/ma_grads.h, group by group."""
    rows, cols = x.shape
    cp, ep = pitches(cols)
    codes = np.zeros((rows, cp), np.int8)
    exps = np.zeros((rows, ep), np.uint8)
    for r in range(rows):
        for g in range(cp // 32):
            v = x[r, 32 * g:32 * (g + 1)]
            if not np.all(np.isfinite(v)):
                exps[r, g] = 255
                continue
            top = np.max(np.abs(v)) if v.size else 0.0
            e = -126
            while e < 121 and np.rint(top / 2.0 ** e) > 127:
                e += 1
            codes[r, 32 * g:32 * g + v.size] = np.clip(np.rint(v / 2.0 ** e), -127, 127)
            exps[r, g] = e + 127
    return codes, exps


def unpack(codes, exps, cols):
    e = exps[:, :codes.shape[1] // 32].astype(np.int64)
    s = np.where(e == 255, np.nan, 2.0 ** (np.minimum(e, 254) - 127.0))
    return (codes.astype(np.float64) * np.repeat(s, 32, axis=1))[:, :cols]


def held(x):
    return unpack(*pack(x), x.shape[1])


def rounded(v, tol, out):
    """tol widened by the rounding of v (+- tol) to the output type."""
    return tol + (np.abs(v) + tol) * U[out] + TINY


def embedding_grad(dout, tokens, vocab, scale, pad, old=None):
    """(gradient, float32 error bound): n terms added in any order err by at most
    n u sum|terms|, the scale and its product by 2 u, the old value's sum by u."""
    w = np.zeros((vocab, dout.shape[1]))
    mag = np.zeros_like(w)
    n = np.zeros((vocab, 1))
    for t, v in enumerate(tokens):
        if 0 <= v < vocab and v != pad:
            w[v] += dout[t]
            mag[v] += np.abs(dout[t])
            n[v] += 1
    w *= scale
    tol = (n + 4) * F32 * mag * abs(scale)
    if old is not None:
        w = w + old
        tol = tol + 2 * F32 * (np.abs(w) + np.abs(old))
    return w, tol


def linear_grad(dy, x, old=None):
    """(dY^T X, error bound).  The products are exact; the matrix cores add
    them in float32, each addition off by at most one step (they may cut instead
    of rounding), and a float32 dy makes three products of each: 3 M additions,
    plus those that join partial sums, at most M more."""
    w = dy.T @ x
    mag = np.abs(dy).T @ np.abs(x)
    tol = (4 * dy.shape[0] + 4) * 2 * F32 * mag
    if old is not None:
        w = w + old
        tol = tol + 2 * F32 * (np.abs(w) + np.abs(old))
    return w, tol


def _sig(a):
    e = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


C = 2.0 * np.sqrt(2.0 / np.pi)


def act(kind, g):
    """(act(g), act'(g)) and their absolute error bounds.

    s = 1 / (1 + exp(-a)): a is g (exact) or GELU's polynomial, whose four
    roundings err by 4 u |a|; the exponent's product with log2 e by 2 u |a|
    more (the constant and the product), each times exp's derivative; exp2,
    the sum and the reciprocal by at most 2 + 1 + 2 units.  Below the smallest
    normal float, 2^-126, s may be 0: exp(-a) leaves the range at a = -88.7,
    where s = 2^-128, and the hardware's reciprocal has no denormal results.
    That errs by at most 2^-126 in s, so 2^-126 |g| in act and, with s (1 - s)
    <= s, 2^-126 (1 + |g a'|) in the slope."""
    a = g if kind == "silu" else C * g * (1.0 + 0.044715 * g * g)
    s = _sig(a)
    da = np.ones_like(g) if kind == "silu" else C * (1.0 + 3 * 0.044715 * g * g)
    rel = (6 * np.minimum(np.abs(a), 200.0) + 8) * F32
    p = _sig(a) * _sig(-a)
    slope = s + p * g * da
    # slope = s + s (1 - s) g a': 1 - s errs by rel s, absolutely
    slope_tol = s * rel + np.abs(g * da) * (p * (2 * rel + 8 * F32) + s * s * rel)
    return (g * s, slope, (rel + 2 * F32) * np.abs(g * s) + UNDER * np.abs(g),
            slope_tol + 4 * F32 * np.abs(slope) + UNDER * (1 + np.abs(g * da)))
