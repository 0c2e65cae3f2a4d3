"""Plain 64-bit forms of the 4-bit cache, its attention, the accumulated attention weight and the eviction,
written from the definitions in include/tls.h (numpy; no code of the library)."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # unit roundoff of fp32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([(b & 7) * 2.0 ** -17 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 15) for b in range(0xE3)])


def nearest(x, table):
    """Index of the nearest value of an ascending table, ties to the even index."""
    lo = np.clip(np.searchsorted(table, x, side="right") - 1, 0, len(table) - 2)
    below, above = x - table[lo], table[lo + 1] - x
    return lo + ((above < below) | ((above == below) & (lo % 2 == 1)))


def quantise(x):
    """fp64 rows [..., d] -> (magnitude codes with sign bit [..., d], scale bytes [..., d / 16])."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16)
    amax = np.abs(g).max(-1)
    fine = np.isfinite(g).all(-1)
    b = np.where(fine, nearest(np.where(fine, amax, 0) / 6, SCALES), 0xFF)
    s = np.where(fine, SCALES[np.where(fine, b, 0)], 0)[..., None]
    on = np.broadcast_to(s > 0, g.shape)
    y = np.divide(np.abs(g), s, out=np.zeros_like(g), where=on)
    m = np.where(on, nearest(np.where(on, y, 0), GRID), 0)
    code = np.where(on, m | (np.signbit(g).astype(np.int64) << 3), 0)
    return code.reshape(x.shape), b.astype(np.uint8)


def value(code, b):
    """The numbers that codes [..., d] and scale bytes [..., d / 16] stand for."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(b == 0xFF, np.nan, SCALES[np.minimum(b, 0xE2)])
    return (v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16) * s[..., None]).reshape(v.shape)


def split(rec, d):
    """Records uint8 [..., 9 d / 8] -> (K, V) in fp64."""
    def codes(c):
        return np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], 2 * c.shape[-1]).astype(np.int64)

    h, s = d // 2, d // 16
    return (value(codes(rec[..., :h]), rec[..., h:h + s]),
            value(codes(rec[..., h + 2 * s:]), rec[..., h + s:h + 2 * s]))


def records(K, V):
    """fp64 rows -> records uint8 [..., 9 d / 8]."""
    def pack(c):
        return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)

    kc, ks = quantise(K)
    vc, vs = quantise(V)
    return np.concatenate((pack(kc), ks, vs, pack(vc)), -1)


def attention(q, K, V, tokens, scale):
    """One group: q [G, d], K, V [n, d], token ids (repeats count twice).  (out, lse, bound on |out|'s and on
    lse's error of an fp32 evaluation).

    The bound: a score is a sum of d exact products, so any order of fp32 additions is off by at most
    (d + 2) u sum|q k|, doubled for a tensor core's truncating alignment, and its scaling and exponent add a
    few u |s|.  A weight exp(s - m) is then off by that much relatively (to both sides of the quotient:
    twice), plus 2^-20 for exp2, the two-part fp16 weight and the fp32 sums over the tokens' partials.
    Small weights: the fp16 parts hold w 2^14 / w_max or more, and an fp16 number below 2^-14 is off by at most
    half its step of 2^-24.  So each weight may be off by 2^-25 2^-14 = 2^-39 of the largest, which adds
    2^-39 sum_t |V_t| / z with z = sum_t w_t / w_max (the sum z itself is of unrounded weights)."""
    q, t = np.asarray(q, np.float64), np.asarray(tokens, np.int64)
    if len(t) == 0:
        z = np.zeros((len(q), V.shape[1]))
        return z, np.full(len(q), -np.inf), z + 1e-30, np.zeros(len(q))
    k, v = K[t], V[t]
    s = q @ k.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    z = p.sum(1, keepdims=True)
    ds = (2 * (q.shape[1] + 2) * U32 * (np.abs(q) @ np.abs(k).T) * scale + 8 * U32 * (np.abs(s) + 1)).max(1, keepdims=True)
    rel = 2 * ds + 2.0 ** -20 + len(t) * U32
    drop = 2.0 ** -39 * np.abs(v).sum(0) / z
    return (p @ v) / z, (m + np.log(z))[:, 0], rel * ((p @ np.abs(v)) / z) + drop + 1e-30, (rel + 4 * U32 * np.abs(m))[:, 0]


def weights(q, K, lse, tokens, scale, n_ctx):
    """One group's added weights [n_ctx] and a bound on their fp32 error (the scores' as above, a few u of the
    exponent's terms, and u per head of the sum)."""
    q, t = np.asarray(q, np.float64), np.asarray(tokens, np.int64)
    out, tol = np.zeros(n_ctx), np.zeros(n_ctx)
    live = ~np.isneginf(lse)
    if len(t) == 0 or not live.any():
        return out, tol
    q, lse = q[live], np.asarray(lse, np.float64)[live]
    k = K[t]
    s = q @ k.T * scale
    w = np.exp(s - lse[:, None])
    ds = 2 * (q.shape[1] + 2) * U32 * (np.abs(q) @ np.abs(k).T) * scale
    ds = ds + 8 * U32 * (np.abs(s) + np.abs(lse)[:, None] + np.abs(s - lse[:, None]) + 1)
    np.add.at(out, t, w.sum(0))
    np.add.at(tol, t, (w * (ds + 2.0 ** -21)).sum(0) + len(q) * U32 * w.sum(0))
    return out, tol


def keep(w, n, budget, n_sink, n_recent):
    """Ids that stay of one (sequence, KV head), ascending: lexicographic order of (protected, weight, -index)."""
    if n <= budget:
        return np.arange(n)
    t = np.arange(n)
    rank = np.where(np.isnan(w[:n]), -np.inf, w[:n].astype(np.float64))
    guard = (t < n_sink) | (t >= n - n_recent)
    order = np.lexsort((t, -rank, ~guard))  # last key first
    return np.sort(order[:budget])
