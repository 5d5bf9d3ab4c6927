"""fp64 references of the operators around the mixer, from their definitions, and how far
a computation in fp32 with one rounding at the end may be from them.  numpy only."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                          # half a step of fp32, relative
U = {"bf16": 2.0 ** -8, "f32": U32}       # half a step of an output type, relative


def block_norm(o, x, gate, w_post, w_pre, res_scale, eps, sigmoid):
    """(r, y, p): p is what joins the residual.  gate broadcasts against [T, D], or is None."""
    x = np.asarray(x, np.float64)
    p = np.zeros_like(x)
    if o is not None:
        o = np.asarray(o, np.float64)
        n = o
        if w_post is not None:
            n = o / np.sqrt((o * o).mean(-1, keepdims=True) + eps) * np.asarray(w_post, np.float64)
        g = 1.0
        if gate is not None:
            g = np.asarray(gate, np.float64)
            g = 1.0 / (1.0 + np.exp(-g)) if sigmoid else g
        p = res_scale * g * n
    r = x + p
    y = None
    if w_pre is not None:
        y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * np.asarray(w_pre, np.float64)
    return r, y, p


def block_norm_bounds(r, y, p):
    """Bounds on the errors of r and y before their last rounding.

    A sum of squares over a row adds at most 32 terms in a thread, then 5 levels in a warp
    and 16 warps: off by at most 53 U32, half of that after the square root, and 3 U32 for
    rsqrt (2 ulp), the mean and eps.  exp in the sigmoid: 2 ulp and an argument rounded
    twice, |g| <= 8 in the tests: 2 * 8 * 1.5 U32 + 4 U32; the quotient and its sum 3 U32.
    Five products: 5 U32.  In all below 128 U32 = 2^-17 of p, and U32 of the sum r; y takes
    r's error, its effect on the row's mean square, and a norm's 40 U32."""
    e_r = 2.0 ** -17 * np.abs(p) + U32 * np.abs(r)
    if y is None:
        return e_r, None
    norm = np.sqrt((r * r).sum(-1, keepdims=True))
    row = np.sqrt((e_r * e_r).sum(-1, keepdims=True)) / np.maximum(norm, 1e-300)
    with np.errstate(divide="ignore", invalid="ignore"):
        per = np.where(r != 0, np.abs(y / r), 0.0)
    return e_r, per * e_r + np.abs(y) * (row + 40 * U32)


def quantize_rows(x):
    """(q as fp64, scale): exact for bf16 rows (127 x is exact, and fp64 resolves every tie)."""
    x = np.asarray(x, np.float64)
    amax = np.abs(x).max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(127.0 * x / amax)
    return np.where(amax > 0, q, 0.0), amax[..., 0] / 127.0


def linear_i8(q, q_scale, w, w_scale):
    """The exact int64 sums times both scales, in fp64.  fp32 converts the sum, multiplies the
    scales and multiplies the two: 3 roundings."""
    acc = np.asarray(q, np.int64) @ np.asarray(w, np.int64).T
    return acc * (np.asarray(q_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :])


I8_ERR = 3.01 * U32   # of |y|, before its last rounding


def log_softmax(x):
    x = np.asarray(x, np.float64)
    m = x.max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        return x - m - np.log(np.exp(x - m).sum(-1, keepdims=True))


# What a sum of exponentials is off by, relative to itself, and so the log-sum-exp absolutely:
# * 2^y by ex2.approx: 2^-22 = 4 U32.
# * Its argument y = x log2(e) - c, one fused operation: the terms that matter have |y| < 32 (the
#   largest of a lane's lies between -1 and 32, kSpan, above its c), so half a step is
#   2^-20, times ln 2: 11.1 U32.  About the top itself (large logits) it is (x - top) log2(e),
#   two roundings of 2 U32 d nats together at the distance d; 2^20 logits at one distance
#   have the share 2^20 e^-d / (1 + 2^20 e^-d) of the sum, and d times that is at most 10.5:
#   21 U32.
# * log2(e) in fp32, off by 1.34e-8, scales those distances: 10.5 * 1.34e-8 = 2.4 U32.
# * fp32 additions before a sum goes to fp64: chains of 8 (bf16; 4 in fp32) in four sums, joined in
#   two more: 7 + 2 = 9 U32; about the top itself 7.
# 4 + 11.1 + 2.4 + 9 = 27 U32 = 1.6e-6, and 4 + 21 + 2.4 + 7 = 35 U32 = 2.1e-6 about the top itself;
# the rest is in fp64.  Below 2.5e-6; twice that is allowed.  The published scores are rounded to
# fp32 besides.
BEAM_ERR = 5e-6


def beam_select(logits, scores, n, finished=None, pad=0):
    """Per group (parents, tokens, scores), and the smallest difference between successive
    results of different beams (the first left out among them)."""
    G, W, V = logits.shape
    parents, tokens = np.full((G, n), -1, np.int32), np.full((G, n), -1, np.int32)
    best = np.full((G, n), -np.inf)
    gap = np.inf
    for g in range(G):
        s = np.asarray(scores[g], np.float64)[:, None] + log_softmax(logits[g])
        if finished is not None:
            for w in np.nonzero(finished[g])[0]:
                s[w] = -np.inf
                s[w, pad] = scores[g, w]
        flat = np.where(np.isfinite(s), s, -np.inf).reshape(-1)
        k = min(n + 1, flat.size)
        cut = np.partition(flat, flat.size - k)[flat.size - k]
        at = np.nonzero((flat >= cut) & (flat > -np.inf))[0]
        at = at[np.lexsort((at, -logits[g].reshape(-1)[at], at // V, -flat[at]))]   # (a beam's own by their logits)
        for a, b in zip(at[:n], at[1:n + 1]):
            if a // V != b // V and flat[a] != flat[b]:
                gap = min(gap, flat[a] - flat[b])
        at = at[:n]
        parents[g, :len(at)], tokens[g, :len(at)], best[g, :len(at)] = at // V, at % V, flat[at]
    return parents, tokens, best, gap


def reorder(state, parents):
    """state [G * W, ...] -> the same after slot w of group g took slot parents[g, w]."""
    G, W = parents.shape
    own = np.arange(W)[None, :].repeat(G, 0)
    at = np.where(parents < 0, own, parents) + np.arange(G)[:, None] * W
    return state[at.reshape(-1)]
