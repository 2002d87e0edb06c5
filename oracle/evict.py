"""The attention weight of cached keys and eviction by it, in plain fp64 NumPy from
the definitions (test infrastructure only).

Weights: key j of a cache head gets the sum of exp(scale q k_j - LSE) over the rows of
its query heads that see it, on top of what it had if it is older than start[b].

Eviction: a cache head of a sequence keeps its first `sink` tokens, its last `recent`
and of the others those of the largest weight (a NaN below all others, the lower
position first among equals), n = min(len, keep) in all, in their order. A page that
changes gets the smallest scale 2^k >= 2^-100 with absmax <= 448 * 2^k over its tokens;
K codes that are NaN, and tokens whose K or V scale is no scale (negative, infinite,
NaN), do not count and become NaN keys and, the latter, zero values.
"""
from __future__ import annotations

import numpy as np

from .cache import PAGE, scale_exponent
from .fp8 import e4m3_round


def weigh(q, k8, kscale, table, lens, q_lens, lse, weights, start, scale, causal=True, lts=None,
          lte=None, uts=None, ute=None):
    """(weights [pages, Hk, 64], tol): the result and, for error bounds, sum over rows of
    p * (the row's error in units of its weight), see below; also rows counted."""
    B, H, N, d = q.shape
    Hk = k8.shape[1]
    w, tol = np.array(weights, np.float64), np.zeros(weights.shape)
    bounds = [x for x in ((lts, lte), (uts, ute)) if x[0] is not None]
    for b in range(B):
        n, live = int(lens[b]), (N if q_lens is None else int(q_lens[b]))
        first = n - live if start is None else int(start[b])
        pages = [int(p) for p in table[b][:-(-n // PAGE)]]
        i, j = np.arange(n - live, n)[:, None], np.arange(n)[None, :]
        for hk in range(Hk):
            kk = (k8[pages, hk] * np.asarray(kscale, np.float64)[pages, hk][:, None, None]).reshape(-1, d)[:n]
            got, off = np.zeros(n), np.zeros(n)
            for h in range(hk * (H // Hk), (hk + 1) * (H // Hk)):
                hidden = np.zeros((live, n), bool)
                if causal:
                    hidden |= j > i
                for s, e in bounds:
                    hm = h // (H // s.shape[1])
                    hidden |= (s[b, hm, :n][None] <= i) & (i < e[b, hm, :n][None])
                qq = np.asarray(q[b, h, :live], np.float64)
                l = np.asarray(lse[b, h, :live], np.float64)[:, None]
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.where(hidden | np.isneginf(l), 0.0, np.exp(scale * (qq @ kk.T) - l))
                    mag = np.nan_to_num(np.where(hidden, 0.0, scale * (np.abs(qq) @ np.abs(kk).T)))
                    # a score's error (as in the attention's bounds), LSE in log2 units, the
                    # exponential, and a chain of one addition a row
                    err = 2 * (mag * 2.0 ** -18 + 2.0 ** -20) + np.abs(np.nan_to_num(l)) * 2.0 ** -21 + \
                        2.0 ** -19 + live * (H // Hk) * 2.0 ** -24
                    got += p.sum(0)
                    off += (np.nan_to_num(p) * err).sum(0) + live * 2e-38
            at = [(pages[t // PAGE], hk, t % PAGE) for t in range(n)]
            for t in range(n):
                old = w[at[t]] if t < first else 0.0
                w[at[t]] = old + got[t]
                tol[at[t]] = off[t] + abs(old) * 2.0 ** -23 + abs(got[t]) * 2.0 ** -23
    return w, tol


def kept(weights, n, keep, sink, recent):
    """Positions, in order, of the tokens that a head of n tokens with these weights keeps."""
    m = min(n, max(int(keep), 0))
    first = min(sink, m)
    last = min(recent, m - first)
    middle = list(range(first, n - last)) if m < n else []
    w = np.asarray(weights, np.float64)
    key = lambda t: (np.isnan(w[t]), -w[t] if not np.isnan(w[t]) else 0.0, t)
    if m == n:
        return list(range(n))
    chosen = sorted(sorted(middle, key=key)[:m - first - last])
    return list(range(first)) + chosen + list(range(n - last, n))


def no_scale(s):
    return not (np.isfinite(s) and s >= 0)


def evict(k8, kscale, v8, vscale, weights, table, lens, keep, sink, recent, out_table=None):
    """The cache afterwards, as (K values of codes, scales, V, scales, weights, kept
    positions [b][hk]). out_table None: in place."""
    k8, v8 = np.array(k8, np.float64), np.array(v8, np.float64)
    kscale, vscale = np.array(kscale, np.float64), np.array(vscale, np.float64)
    src = [x.copy() for x in (k8, kscale, v8, vscale)]
    w = np.array(weights, np.float64)
    w_src = w.copy()
    places = []
    for b in range(len(lens)):
        n = int(lens[b])
        places.append([])
        for h in range(k8.shape[1]):
            pages = [int(p) for p in table[b][:-(-n // PAGE)]]
            ww = w_src[pages, h].reshape(-1)[:n] if n else np.zeros(0)
            pos = kept(ww, n, keep[b], sink, recent)
            places[-1].append(pos)
            for dp in range(-(-len(pos) // PAGE)):
                mine = pos[dp * PAGE:(dp + 1) * PAGE]
                if out_table is None and mine == list(range(dp * PAGE, dp * PAGE + len(mine))):
                    continue  # every token stays where it is
                to = int((table if out_table is None else out_table)[b][dp])
                kk = np.stack([src[0][pages[t // PAGE], h, t % PAGE] for t in mine])
                vv = np.stack([src[2][pages[t // PAGE], h, :, t % PAGE] for t in mine])
                ks = np.array([src[1][pages[t // PAGE], h] for t in mine])
                vs = np.array([src[3][pages[t // PAGE], h] for t in mine])
                bad = np.array([no_scale(a) or no_scale(z) for a, z in zip(ks, vs)])
                for x, s, codes, scales, key in ((kk, ks, k8, kscale, True), (vv, vs, v8, vscale, False)):
                    nan = np.isnan(x) | bad[:, None]
                    y = np.where(nan, 0.0, x) * np.where(bad, 1.0, s)[:, None]
                    s_new = 2.0 ** scale_exponent(np.abs(y).max())
                    y = e4m3_round(y / s_new)
                    y = np.where(nan, np.nan if key else 0.0, y)
                    page = np.zeros((PAGE, x.shape[1]))
                    page[:len(mine)] = y
                    codes[to, h] = page if key else page.T
                    scales[to, h] = s_new
                w[to, h] = 0.0
                w[to, h, :len(mine)] = [w_src[pages[t // PAGE], h, t % PAGE] for t in mine]
    return k8, kscale, v8, vscale, w, places
