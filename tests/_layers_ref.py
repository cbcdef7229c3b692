"""The layer operators' definitions in float64 NumPy, and the error bounds their
float32 arithmetic keeps, for the tests of include/ma_layers.h.

A rounding to a type errs by at most half a step, U[type] relative to the
value.  `tol` arrays are absolute bounds per element."""

import numpy as np

from tests._grads_ref import F32, TINY, U, UNDER


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


def _attend(q, k, scale, causal):
    """(scores, mask of what is seen, bound of the scores): one head of one sequence.  A product of d
    terms is summed by the matrix cores in float32, each addition off by at most one step (they may
    cut instead of rounding), from exact products of bfloat16 and rounded ones of float32; scale and the
    softmax's arguments by 6 u of the score."""
    n, m = q.shape[0], k.shape[0]
    z = scale * (q @ k.T)
    seen = np.ones((n, m), bool)
    if causal:
        seen = np.arange(m)[None] <= np.arange(n)[:, None] + m - n
    tol = scale * (2 * q.shape[1] + 4) * 2 * F32 * (np.abs(q) @ np.abs(k).T) + 6 * F32 * np.abs(z)
    return z, seen, tol


def _packed(cu_q, cu_k, heads, kv_heads):
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        for h in range(heads):
            yield slice(a, b), slice(c, d), h, h // (heads // kv_heads)


def attention(q, k, v, cu_q, cu_k, causal, scale, kind):
    """(o, lse, bounds before rounding; NaN where no sequence is).  The probabilities of a
    bfloat16 call are rounded once more for their product with v."""
    up = U[kind] if kind == "bf16" else 0.0
    o, lse = np.full(q.shape, np.nan), np.full((q.shape[1], q.shape[0]), np.nan)
    otol, ltol = np.zeros(q.shape), np.zeros(lse.shape)
    for a, b, h, g in _packed(cu_q, cu_k, q.shape[1], k.shape[1]):
        z, seen, zt = _attend(q[a, h], k[b, g], scale, causal)
        n, m = z.shape
        if n == 0:
            continue
        if m == 0:
            o[a, h], lse[h, a] = 0.0, -np.inf
            continue
        z = np.where(seen, z, -np.inf)
        top = np.max(z, 1, keepdims=True)
        none = np.isneginf(top[:, 0])
        e = np.exp(z - np.where(np.isneginf(top), 0.0, top))
        s = e.sum(1)
        p = e / np.where(none, 1.0, s)[:, None]
        # (the reference of the exponent may be 2^8 below the top: 8 ln 2 more in its argument)
        zt = np.where(seen, zt, 0.0) + 6 * F32 * np.where(p > 0, np.abs(z - np.where(seen, top, 0.0)) + 6, 0.0) * seen
        o[a, h] = p @ v[b, g]
        lse[h, a] = np.where(none, -np.inf, np.where(none, 0.0, top[:, 0]) + np.log(np.where(none, 1.0, s)))
        mean = (p * zt).sum(1, keepdims=True) + (m + 8) * F32
        otol[a, h] = (p * (zt + mean + up * (1 + 2.0 ** -8) + (2 * m + 8) * F32)) @ np.abs(v[b, g])
        otol[a, h] += (seen * UNDER) @ np.abs(v[b, g])
        ltol[h, a] = mean[:, 0] + 4 * F32 * (np.abs(np.where(none, 0, lse[h, a])) + np.abs(np.where(none, 0, top[:, 0])))
    return o, lse, otol, ltol


def attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal, scale, kind):
    """(dq, dk, dv, their bounds before rounding; NaN where no sequence is).  A probability below
    2^-126, the smallest normal float, may be 0 (the hardware's 2^x and matrix instructions have no
    denormal results), and so may a score's gradient: an absolute 2^-126 of each, times what it
    is multiplied with (with |dp - delta| of 30, queries of 8 and 400 terms up to 1e-33)."""
    up = U[kind] * (1 + 2.0 ** -8) if kind == "bf16" else 0.0
    res = [np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(v.shape, np.nan)]
    tol = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    for x, cu in zip(res, (cu_q, cu_k, cu_k)):
        for a, b in zip(cu, cu[1:]):
            x[a:b] = 0.0
    d2 = 2 * q.shape[2] + 8
    for a, b, h, g in _packed(cu_q, cu_k, q.shape[1], k.shape[1]):
        z, seen, zt = _attend(q[a, h], k[b, g], scale, causal)
        n, m = z.shape
        if n == 0 or m == 0:
            continue
        L = lse[h, a][:, None]
        none = np.isneginf(L)
        p = np.where(seen & ~none, np.exp(z - np.where(none, 0.0, L)), 0.0)
        rel = zt + 6 * F32 * (np.abs(np.where(none, 0.0, L)) + np.abs(z) + 2)
        dh, oh = do[a, h], o[a, h]
        delta = (dh * oh).sum(1, keepdims=True)
        dt = d2 * F32 * (np.abs(dh) * np.abs(oh)).sum(1, keepdims=True)
        dp = dh @ v[b, g].T
        pt = d2 * 2 * F32 * (np.abs(dh) @ np.abs(v[b, g]).T)
        ds = p * (dp - delta)
        st = np.abs(ds) * (rel + up + 3 * F32) + p * (pt + dt + 2 * F32 * (np.abs(dp) + np.abs(delta)))
        st += seen * UNDER * (np.abs(dp) + np.abs(delta) + 1)
        res[0][a, h] += scale * ds @ k[b, g]
        tol[0][a, h] += scale * (st + (2 * m + 8) * F32 * np.abs(ds)) @ np.abs(k[b, g])
        more = (2 * n * (q.shape[1] // k.shape[1]) + 8) * F32
        res[1][b, g] += scale * ds.T @ q[a, h]
        tol[1][b, g] += scale * (st + more * np.abs(ds)).T @ np.abs(q[a, h])
        res[2][b, g] += p.T @ dh
        tol[2][b, g] += (p * (rel + up + more) + seen * UNDER).T @ np.abs(dh)
    return res, tol
