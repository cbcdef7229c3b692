"""The layer operators' definitions in float64 NumPy, and the error bounds their
float32 arithmetic keeps, for the tests of include/ma_layers.h.

A rounding to a type errs by at most half a step, U[type] relative to the
value.  `tol` arrays are absolute bounds per element."""

import numpy as np

from tests._grads_ref import F32, TINY, U


def rms_norm(x, w, res=None, eps=1e-6, off=0.0):
    """(y, s, inv, bound of y, of s, of inv before they are rounded to an array's
    type).  A sum of n squares errs by at most n u of itself (n / 2 in the root), the
    mean's product, eps and the root by 4 u, and y's two products and w + off by 3 u more;
    x + res, the only place where something cancels, by u of the sum."""
    s = x if res is None else x + res
    n = x.shape[1]
    inv = 1.0 / np.sqrt(np.mean(s * s, 1) + eps)
    y = s * inv[:, None] * (w + off)
    ds = np.zeros_like(s) if res is None else F32 * np.abs(s)
    di = inv * F32 * (n / 2 + 6)
    dy = np.abs(y) * F32 * (n / 2 + 12) + np.abs(s * inv[:, None]) * F32 * (np.abs(w) + abs(off))
    return y, s, inv, dy, ds, di


def rms_norm_backward(dy, s, inv, w, off=0.0, dsum=None, dw=None):
    """(ds, dw, bounds).  The mean of g h errs by n + 4 roundings of its terms' magnitudes,
    every other value by a few of its own; a sum over rows by as many roundings as it has
    rows."""
    n = s.shape[1]
    h = s * inv[:, None]
    g = dy * (w + off)
    dot = np.mean(g * h, 1, keepdims=True)
    mag = np.mean(np.abs(g * h), 1, keepdims=True)
    dg = np.abs(dy) * F32 * 2 * (np.abs(w) + abs(off))
    ds = inv[:, None] * (g - h * dot)
    tol = np.abs(inv[:, None]) * (dg + 4 * F32 * (np.abs(g) + np.abs(h * dot)) + np.abs(h) * (n + 8) * F32 * mag)
    tol += np.abs(inv[:, None]) * np.abs(h) * np.mean(np.abs(h) * dg, 1, keepdims=True)
    if dsum is not None:
        ds = ds + dsum
        tol = tol + F32 * np.abs(ds)
    out = np.sum(dy * h, 0)
    wtol = (s.shape[0] + 4) * F32 * np.sum(np.abs(dy * h), 0)
    if dw is not None:
        out = out + dw
        wtol = wtol + 2 * F32 * (np.abs(out) + np.abs(dw))
    return ds, out, tol, wtol


def rotary_table(sections, theta, order, restart):
    """[(axis, frequency)] of every pair."""
    left, out = list(sections), []
    total = sum(sections)
    while sum(left):
        for a in range(len(left)):
            for _ in range(left[a] if order == "blocks" else min(1, left[a])):
                j = sections[a] - left[a]
                left[a] -= 1
                out.append((a, theta ** (-j / sections[a] if restart else -len(out) / total)))
    return out


def rotary(x, pos, table, layout, inverse=False):
    """(turned x, bound before rounding) of x (tokens, heads, dim) and pos (axes, tokens).  Sine
    and cosine err by 2^-22 (their library's 2 u, and u of the remainder in turns, times pi);
    the two products and their sum by 3 u of their magnitudes."""
    out, tol = x.copy(), np.zeros_like(x)
    pairs = len(table)
    for i, (a, f) in enumerate(table):
        ang = np.asarray(pos[a], np.float64) * f * (-1 if inverse else 1)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        p, q = (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)
        u, v = x[:, :, p], x[:, :, q]
        out[:, :, p], out[:, :, q] = u * c - v * s, u * s + v * c
        # (NumPy's own angle errs by 2^-53 of itself, and so does ours)
        t = (np.abs(u) + np.abs(v)) * (2.0 ** -22 + 3 * F32 + np.abs(ang)[:, None] * 2.0 ** -51)
        tol[:, :, p] = tol[:, :, q] = t
    return out, tol


def rounded(v, tol, out):
    """tol widened by the rounding of v (+- tol) to the output type."""
    return tol + (np.abs(v) + tol) * U[out] + TINY


def logprob(z, ids, scale, top=0):
    """(logprob, entropy, lse, ids, top's logprobs, bounds of the five float results): rows of
    z (tokens, vocab).

    With u = (z - m) k, k = scale log2 e rounded, e = 2^u: u errs by 4 u' |u| (u' = 2^-24: the
    difference, k, the product), so e by (3 |u| + 2) u' of itself (2^x's own error is one step),
    and a sum of n terms in pieces by at most n / 8 + 40 roundings more (threads take at least 8
    elements each in turn; short rows fewer).  The absolute error of ln s is that relative error
    averaged with weights p, of t / s the same with |u| more.  lse and the products with scale
    add a few u' of their magnitudes."""
    n, v = z.shape
    zs = z * scale
    m = np.max(zs, 1, keepdims=True)
    none = np.isneginf(m[:, 0])
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        d = zs - m
        e = np.exp(d)
        s = e.sum(1)
        ls = np.log(s)
        lse = np.where(none, -np.inf, m[:, 0] + ls)
        p = np.where(none[:, None], 0.0, e / np.maximum(s, 1e-300)[:, None])
        far = np.where(p > 0, -d, 0.0)                    # ln units, at least 0
        ent = np.where(none, 0.0, np.log(np.maximum(s, 1e-300)) + (p * far).sum(1))
    rel = (p * (5 * far + 3)).sum(1) * F32 + (v / 8 + 40) * F32
    ls_tol = rel + 2 * F32 * np.abs(np.log(np.maximum(s, 1e-300)))
    lse_tol = ls_tol + 3 * F32 * (np.abs(m[:, 0]) + np.abs(np.where(none, 0, lse)))
    ent_tol = 2 * ls_tol + (p * far * (5 * far + 6)).sum(1) * F32 + (v / 8 + 44) * F32 * ((p * far).sum(1) + ent)
    ok = (ids >= 0) & (ids < v)
    at = np.where(ok, ids, 0)
    rows = np.arange(n)
    # (from the differences: far values less their lse would cancel even in 64 bits)
    with np.errstate(invalid="ignore"):
        lp = np.where(ok, np.where(none, -np.inf, d[rows, at] - ls), 0.0)
    dist = np.abs(np.where(np.isfinite(zs), d, 0.0))
    lp_tol = ls_tol + 4 * F32 * (dist[rows, at] + np.abs(np.where(np.isfinite(lp), lp, 0)))
    best = np.lexsort((np.broadcast_to(np.arange(v), z.shape), -z), axis=1)[:, :top]
    with np.errstate(invalid="ignore"):
        tl = np.where(none[:, None], -np.inf, np.take_along_axis(d, best, 1) - ls[:, None])
    tl_tol = ls_tol[:, None] + 4 * F32 * (np.take_along_axis(dist, best, 1) + np.abs(np.where(np.isfinite(tl), tl, 0)))
    return (lp, ent, lse, best, tl), (lp_tol, ent_tol, lse_tol, None, tl_tol)


def logprob_backward(z, ids, scale, lse, g, ent=None, h=None):
    """(dlogits, bound before rounding).  log p = z scale - lse errs by 2 u' of itself and u'
    of the product's rounded input, so p by 3 u' |log p| + 2 u'; the rest is a few u'."""
    none = np.isneginf(lse)
    with np.errstate(invalid="ignore"):
        lp = z * scale - np.where(none, 0.0, lse)[:, None]
    p = np.where(none[:, None], 0.0, np.exp(lp))
    far = np.where(p > 0, np.where(np.isfinite(lp), lp, 0.0), 0.0)
    h0 = np.zeros_like(g) if h is None else h
    e0 = np.zeros_like(g) if ent is None else ent
    ok = (ids >= 0) & (ids < z.shape[1]) & ~none
    g1 = np.where((ids >= 0) & (ids < z.shape[1]), g, 0.0)
    c = g1[:, None] + h0[:, None] * (far + e0[:, None])
    d = -p * c
    rows = np.arange(len(ids))[ok]
    d[rows, ids[ok]] += g[ok]
    mag = np.abs(g1)[:, None] + np.abs(h0)[:, None] * (np.abs(far) + np.abs(e0)[:, None])
    tol = p * mag * F32 * (4 * np.abs(far) + 10)
    tol[rows, ids[ok]] += 3 * F32 * np.abs(g[ok])
    return d * scale, tol * scale
