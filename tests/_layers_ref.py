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
