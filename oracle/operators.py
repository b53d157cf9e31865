"""Float64 oracle of the operators around the layer (test infrastructure).

Written from the formulas in ``include/lmoe.h`` with explicit loops over
tokens where that is the plainest form; shares no code with the library.
Inputs are float arrays holding the exact values the kernels read.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _clean(l):
    l = np.asarray(l, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, np.float64(np.finfo(np.float32).max))


def route_scores(l, softmax: bool):
    """Scores [T, E] of cleaned logits; 0 where the logit is -inf."""
    l = _clean(l)
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        on = l[t] > -np.inf
        if not on.any():
            continue
        v = l[t][on]
        with np.errstate(over="ignore"):
            if softmax:
                e = np.exp(v - v.max())
                s[t][on] = e / e.sum()
            else:
                s[t][on] = 1.0 / (1.0 + np.exp(-v))
    return s


def route(l, bias, K, softmax=False, n_group=1, topk_group=1, group_score=2, renorm=True,
          scale=1.0):
    """(idx [T, K] ascending, w [T, K], gap [T]): gap is the distance, in
    biased score (or logit, without a bias), at the border that decided the
    selection; inf where nothing was left out."""
    s = route_scores(l, softmax)
    l = _clean(l)
    T, E = l.shape
    on = l > -np.inf
    b = np.where(on, s + (0.0 if bias is None else np.asarray(bias, np.float64)), -np.inf)
    order = b if bias is not None else l
    idx = np.zeros((T, K), np.int64)
    w = np.zeros((T, K))
    G = E // n_group
    for t in range(T):
        allowed = list(range(E))
        if n_group > 1:
            gs = [np.sort(b[t, g * G:(g + 1) * G])[::-1][:group_score].sum()
                  for g in range(n_group)]
            kept = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            allowed = [e for g in sorted(kept) for e in range(g * G, (g + 1) * G)]
        chosen = sorted(sorted(allowed, key=lambda e: (-order[t, e], e))[:K])
        idx[t] = chosen
        p = s[t, chosen]
        w[t] = scale * p / (p.sum() + 1e-20) if renorm else scale * p
    return idx, w


def route_backward(l, idx, dw, softmax=False, renorm=True, scale=1.0):
    """(dlogits, magnitude): magnitude is the same sum with absolute values
    of its terms, the scale of the rounding errors of each element."""
    s = route_scores(l, softmax)
    T, E = s.shape
    dl, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ids = [int(i) for i in idx[t]]
        ok = [0 <= i < E for i in ids]
        p = np.array([s[t, i] if o else 0.0 for i, o in zip(ids, ok)])
        g = np.where(ok, np.asarray(dw[t], np.float64), 0.0) * scale
        if renorm:
            S = p.sum() + 1e-20
            dp = (g - (g * p).sum() / S) / S
            mp = (np.abs(g) + (np.abs(g) * p).sum() / S) / S
        else:
            dp, mp = g, np.abs(g)
        ds, ms = np.zeros(E), np.zeros(E)
        for i, o, a, m in zip(ids, ok, dp, mp):
            if o:
                ds[i] += a
                ms[i] += m
        if softmax:
            # renormalised, sum ds s = D / S (1 - P / S) with D = sum g p and
            # P = S - 1e-20: taken as D / S * 1e-20 / S, since the difference of
            # the two nearly equal sums would leave 1e-17 of rounding here
            c = (g * p).sum() / S * (1e-20 / S) if renorm else (ds * s[t]).sum()
            dl[t] = s[t] * (ds - c)
            mc = (np.abs(g) * p).sum() / S * (1e-20 / S) if renorm else (ms * s[t]).sum()
            mag[t] = s[t] * (ms + mc)
        else:
            lt = _clean(l[t:t + 1])[0]
            e = np.exp(-np.abs(np.where(lt > -np.inf, lt, 0.0)))
            slope = np.where(lt > -np.inf, e / (1.0 + e) ** 2, 0.0)
            dl[t], mag[t] = ds * slope, ms * slope
    return dl, mag


def _f64(v):
    return None if v is None else np.asarray(v, np.float64)


def block_norm(h, y, pre, post, gate, alpha, eps):
    """(h_out, x or None, ry, rh); gate [D], [T, 1] or [T, D] or None."""
    h, y, pre, post, gate, alpha = (_f64(v) for v in (h, y, pre, post, gate, alpha))
    T, D = h.shape
    y = np.zeros_like(h) if y is None else y
    ry = np.ones((T, 1))
    n = y
    if post is not None:
        ry = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        n = post * y * ry
    h2 = (1.0 if alpha is None else alpha) * h + (1.0 if gate is None else gate) * n
    if pre is None:
        return h2, None, ry, np.ones((T, 1))
    rh = 1.0 / np.sqrt((h2 * h2).mean(1, keepdims=True) + eps)
    return h2, pre * h2 * rh, ry, rh


def block_norm_backward(h, y, dh_out, dx, pre, post, gate, alpha, eps):
    """{name: (gradient, magnitude)}; magnitude bounds the sum of the absolute
    values of the terms of each element."""
    h, y, pre, post, gate, alpha, dh_out, dx = (
        _f64(v) for v in (h, y, pre, post, gate, alpha, dh_out, dx))
    T, D = h.shape
    h2, _, ry, rh = block_norm(h, y, pre, post, gate, alpha, eps)
    yv = np.zeros_like(h) if y is None else y
    a1 = 1.0 if alpha is None else alpha
    g1 = 1.0 if gate is None else gate
    p1 = 1.0 if post is None else post
    yn = yv * ry
    n = p1 * yn
    mh2 = np.abs(a1 * h) + np.abs(g1 * n)
    G = np.zeros_like(h) if dh_out is None else dh_out.copy()
    M = np.abs(G)
    out = {}
    if dx is not None:
        hn, mhn = h2 * rh, mh2 * rh
        a = pre * dx
        G = G + rh * (a - hn * (a * hn).mean(1, keepdims=True))
        M = M + rh * (np.abs(a) + mhn * (np.abs(a) * mhn).mean(1, keepdims=True))
        out["dpre_weight"] = ((dx * hn).sum(0), (np.abs(dx) * mhn).sum(0))
    elif pre is not None:
        out["dpre_weight"] = (np.zeros(D), np.zeros(D))
    out["dh"] = (a1 * G, np.abs(a1) * M)
    if alpha is not None:
        out["dres_scale"] = ((G * h).sum(0), (M * np.abs(h)).sum(0))
    dn, mdn = g1 * G, np.abs(g1) * M
    if post is not None:
        out["dpost_weight"] = ((dn * yn).sum(0), (mdn * np.abs(yn)).sum(0))
    if y is not None:
        if post is None:
            out["dy"] = (dn, mdn)
        else:
            b, mb = p1 * dn, np.abs(p1) * mdn
            out["dy"] = (ry * (b - yn * (b * yn).mean(1, keepdims=True)),
                         ry * (mb + np.abs(yn) * (mb * np.abs(yn)).mean(1, keepdims=True)))
    if gate is not None:
        d, m = G * n, M * np.abs(n)
        if gate.ndim == 1:
            d, m = d.sum(0), m.sum(0)
        elif gate.shape == (T, 1) and D != 1:
            d, m = d.sum(1, keepdims=True), m.sum(1, keepdims=True)
        out["dgate"] = (d, m)
    return out


# ---- 8-bit floating point ------------------------------------------------------


def e4m3_values():
    """The value of each of the 256 e4m3 codes (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return sign * v


def to_e4m3(v):
    """Codes of the e4m3 numbers nearest to v (|v| < 464), ties to even; the
    sign of a value that rounds to zero is kept."""
    v = np.asarray(v, np.float64)
    mags = e4m3_values()[:0x7F]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(mags, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def quantize_fp8(x, block_rows: int = 1):
    """(codes, scales) of x [R, C] fp32, blocks of block_rows x 128; the
    scale and the ratio are the correctly rounded fp32 quotients."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // 128)
    p = np.zeros((rb * block_rows, cb * 128), np.float32)
    p[:R, :C] = x
    p = p.reshape(rb, block_rows, cb, 128)
    scales = np.maximum(np.abs(p).max((1, 3)) / np.float32(E4M3_MAX), np.float32(2.0 ** -126))
    codes = to_e4m3(p / scales[:, None, :, None]).reshape(rb * block_rows, cb * 128)
    return np.ascontiguousarray(codes[:R, :C]), scales


def dequantize(codes, scales, block_rows: int = 1):
    v = e4m3_values()[codes]
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), 128, 1), block_rows, 0)
    return v * s[:v.shape[0], :v.shape[1]]


def fp8_matmul(xc, xs, wc, ws, offsets=None, rows=None):
    """(y, magnitude, written): rows of no group are not written; a row index
    outside x gives zeros."""
    x = dequantize(xc, xs)
    if rows is not None:
        ok = (rows >= 0) & (rows < x.shape[0])
        x = np.where(ok[:, None], x[np.where(ok, rows, 0)], 0.0)
    M = x.shape[0]
    if offsets is None:
        w = dequantize(wc, ws, 128)
        return x @ w.T, np.abs(x) @ np.abs(w).T, np.ones(M, bool)
    N = wc.shape[1]
    y, mag, done = np.zeros((M, N)), np.zeros((M, N)), np.zeros(M, bool)
    for g in range(wc.shape[0]):
        a, b = (min(max(int(o), 0), M) for o in offsets[g:g + 2])
        if b > a:
            w = dequantize(wc[g], ws[g], 128)
            y[a:b], mag[a:b], done[a:b] = x[a:b] @ w.T, np.abs(x[a:b]) @ np.abs(w).T, True
    return y, mag, done


def experts_fp8(z32, idx, w, up, down):
    """The routed experts with FP8 weights and activations: z quantised from
    fp32, the hidden rows relu(.)^2 rounded to fp32 and quantised, fp64 sums.
    ``up[e]`` / ``down[e]``: (codes, scales) of a quantised weight."""
    z = dequantize(*quantize_fp8(z32))
    r = np.zeros_like(z)
    for e in np.unique(idx):
        tok, pos = np.nonzero(idx == e)
        u = z[tok] @ dequantize(*up[int(e)], 128).T
        h = dequantize(*quantize_fp8((np.maximum(u, 0.0) ** 2).astype(np.float32)))
        r[tok] += np.asarray(w, np.float64)[tok, pos][:, None] * (
            h @ dequantize(*down[int(e)], 128).T)
    return r
