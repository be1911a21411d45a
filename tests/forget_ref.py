"""64-bit definitions of the rotary write, the accumulated attention weights and
the eviction, in numpy and straight from their formulas, for the tests."""
from __future__ import annotations

import numpy as np

BT = 16
LOG2E = 1.4426950408889634


def rotate(x, positions, table, pair_axis, interleaved):
    """x [T, H, d]: the pairs of its first rot elements turned, the rest as it is."""
    x = np.asarray(x, np.float64)
    half = table.shape[1] // 2
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        at = positions[pair_axis[i]]
        c, s = (table[at, j].astype(np.float64)[:, None] for j in (i, half + i))
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def rows(cache, table, n, h):
    """The first n rows of KV head h through a table row; cache [NB, Hkv, 16, d]."""
    t = np.arange(n)
    return cache[table[t // BT], h, t % BT]


def weights(q, k, scale, pos):
    """Softmax weights [rows, keys] of query rows q at positions pos over keys 0 .. len(k) - 1."""
    x = (q @ k.T) * scale
    unseen = np.arange(k.shape[0])[None] > np.asarray(pos)[:, None]
    x[unseen] = -np.inf
    x -= x.max(1, keepdims=True)
    e = np.exp(x)
    e[unseen] = 0.0
    w = e / e.sum(1, keepdims=True)
    w[unseen] = 0.0  # no weight, whatever the seen ones hold
    return w


def attention(q, query_start, k_cache, v_cache, tables, lens, scale):
    """[T, Hq, d]: each new token's attention over the tokens up to its own."""
    out = np.zeros(q.shape)
    g = q.shape[1] // k_cache.shape[1]
    for b, n in enumerate(lens):
        lo, hi = int(query_start[b]), int(query_start[b + 1])
        for m in range(q.shape[1] if hi > lo else 0):
            w = weights(q[lo:hi, m], rows(k_cache, tables[b], n, m // g), scale, np.arange(n - (hi - lo), n))
            out[lo:hi, m] = w @ rows(v_cache, tables[b], n, m // g)
    return out


def scores(q, query_start, k_cache, tables, lens, scale, scores_in, window=0):
    """[B, Hkv, S] accumulated weights, NaN where nothing is written.  q [T, Hq, d] and the caches
    as float64; sequence b's new tokens are q rows query_start[b] .. query_start[b + 1]."""
    B, hkv, hq = len(lens), k_cache.shape[1], q.shape[1]
    g = hq // hkv
    S = tables.shape[1] * BT if scores_in is None else scores_in.shape[2]
    out = np.full((B, hkv, S), np.nan)
    for b in range(B):
        lo, hi = int(query_start[b]), int(query_start[b + 1])
        new, n = hi - lo, int(lens[b])
        if n == 0:
            continue
        first = max(0, new - window) if window > 0 else 0
        for h in range(hkv):
            total = np.zeros(n)
            if scores_in is not None:
                total[: n - new] = scores_in[b, h, : n - new]
            if new:
                k = rows(k_cache, tables[b], n, h)
                for m in range(h * g, (h + 1) * g):
                    w = weights(q[lo:hi, m], k, scale, np.arange(n - new, n))
                    total += w[first:].sum(0)
            out[b, h, :n] = total
    return out


def logit_bound(q, k_cache, scale):
    """How far a score weight may be off, relative: fp32 sums of d products for the row's own
    logit and, through its log-sum-exp, for the others', each at most (d + 4) roundings of 2^-23
    of the largest sum of absolute products there can be; plus the exponential's 2^-21."""
    d = q.shape[-1]
    largest = np.sqrt((np.nan_to_num(q) ** 2).sum(-1).max() * (np.nan_to_num(k_cache) ** 2).sum(-1).max())
    return 2 * (d + 4) * 2.0 ** -23 * abs(scale) * largest + 2.0 ** -21


def chosen(score, n, keep, sink, recent):
    """Positions kept of one (sequence, KV head), ascending."""
    m = min(keep, n)
    r = min(recent, m)
    s = min(sink, m - r)
    middle = np.arange(s, n - r)
    key = score[middle].astype(np.float64)
    key = np.where(np.isnan(key), -np.inf, key)
    nan = np.isnan(score[middle])
    order = np.lexsort((middle, nan, -key))  # highest first, then numbers before NaN, then lower positions
    return np.concatenate([np.arange(s), np.sort(middle[order][: m - r - s]), np.arange(n - r, n)]).astype(np.int64)
