"""Rotary positions, the 8-bit paged cache and attention over it, in plain fp64
NumPy from the definitions (test infrastructure only).

Rotation of pair i at position t by a = t f_i: (x, y) -> c (x cos a - y sin a,
y cos a + x sin a), pairs (i, i + n) or (2i, 2i + 1).

Cache: pages of 64 tokens, e4m3 codes with one power-of-two scale per page and
head, the smallest 2^k >= 2^-100 with absmax <= 448 * 2^k over the page's finite
tokens; it only grows while a page fills, and older codes are then rounded
again. A token with a value that is not finite is stored as NaN keys and zero
values and does not count for the scales.
"""
from __future__ import annotations

import math

import numpy as np

from .fp8 import e4m3_round

PAGE = 64


def rope(x, positions, freqs, interleaved=False, mscale=1.0, inverse=False):
    """x [B, H, N, d], positions [B, N], freqs [rot / 2] -> [B, H, N, d]."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    if n == 0:
        return y
    a = np.asarray(positions, np.float64)[:, None, :, None] * np.asarray(freqs, np.float64)
    if inverse:
        a = -a
    first = 2 * np.arange(n) if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    u, w = y[..., first].copy(), y[..., second].copy()
    y[..., first] = mscale * (u * np.cos(a) - w * np.sin(a))
    y[..., second] = mscale * (w * np.cos(a) + u * np.sin(a))
    return y


def scale_exponent(absmax: float) -> int:
    """Smallest k >= -100 with absmax <= 448 * 2^k."""
    if absmax == 0:
        return -100
    k = -100
    m, e = math.frexp(absmax / 1.75)  # absmax <= 1.75 * 2^(8 + k) <=> absmax / 1.75 <= 2^(8 + k)
    k = (e - 1 if m == 0.5 else e) - 8
    return max(k, -100)


def append(k8, kscale, v8, vscale, table, k, v, start, count):
    """The cache after the new tokens, as (K values [pages, Hk, 64, d], scales,
    V values [pages, Hk, d, 64], scales): codes as fp64 values, NaN for a NaN."""
    k8, v8 = np.array(k8, np.float64), np.array(v8, np.float64)
    kscale, vscale = np.array(kscale, np.float64), np.array(vscale, np.float64)
    B, Hk, N, d = k.shape
    for b in range(B):
        n = N if count is None else int(count[b])
        for h in range(Hk):
            for page_i in sorted({(int(start[b]) + t) // PAGE for t in range(n)}):
                page = int(table[b][page_i])
                ts = [t for t in range(n) if (int(start[b]) + t) // PAGE == page_i]
                slots = [(int(start[b]) + t) % PAGE for t in ts]
                begun = slots[0] > 0
                kn, vn = np.asarray(k[b, h, ts], np.float64), np.asarray(v[b, h, ts], np.float64)
                good = np.isfinite(kn).all(1) & np.isfinite(vn).all(1)
                for new, codes, scales, key in ((kn, k8[page, h], kscale, True),
                                                (vn, v8[page, h].T, vscale, False)):
                    top = np.abs(new[good]).max() if good.any() else 0.0
                    s = 2.0 ** scale_exponent(top)
                    if begun:
                        s = max(s, scales[page, h])
                        old = codes[:slots[0]] * (scales[page, h] / s)
                        nan = np.isnan(old)
                        codes[:slots[0]] = np.where(nan, np.nan, e4m3_round(np.where(nan, 0, old)))
                    else:
                        codes[slots[-1] + 1:] = 0.0
                    q = e4m3_round(np.where(good[:, None], new, 0.0) / s)
                    q[~good] = np.nan if key else 0.0
                    codes[slots] = q
                    scales[page, h] = s
    return k8, kscale, v8, vscale


def attend(q, k8, kscale, v8, vscale, table, lens, q_lens, scale, causal=True, lts=None, lte=None,
           uts=None, ute=None):
    """O [B, H, N, d], LSE [B, H, N] and, per row, quantities for error bounds: PV =
    sum_j P_j |V_j| [B, H, N, d], smag = max_j scale sum |q k_j| [B, H, N] and
    top = the number of visible keys times max_j P_j (value scale of j's page)
    [B, H, N]. Rows behind q_lens hold NaN in all of them."""
    B, H, N, d = q.shape
    Hk = k8.shape[1]
    out = [np.full((B, H, N, d), np.nan), np.full((B, H, N), np.nan),
           np.full((B, H, N, d), np.nan), np.full((B, H, N), np.nan), np.full((B, H, N), np.nan)]
    bounds = [x for x in ((lts, lte), (uts, ute)) if x[0] is not None]
    for b in range(B):
        n, live = int(lens[b]), (N if q_lens is None else int(q_lens[b]))
        pages = [int(p) for p in table[b][:-(-n // PAGE)]]
        i = np.arange(n - live, n)[:, None]
        j = np.arange(n)[None, :]
        for h in range(H):
            hk = h // (H // Hk)
            kk = (k8[pages, hk] * np.asarray(kscale, np.float64)[pages, hk][:, None, None]).reshape(-1, d)[:n]
            vv = (v8[pages, hk] * np.asarray(vscale, np.float64)[pages, hk][:, None, None]
                  ).transpose(0, 2, 1).reshape(-1, d)[:n]
            hidden = np.zeros((live, n), bool)
            if causal:
                hidden |= j > i
            for s, e in bounds:
                hm = h // (H // s.shape[1])
                hidden |= (s[b, hm, :n][None] <= i) & (i < e[b, hm, :n][None])
            qq = np.asarray(q[b, h, :live], np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                x = np.where(hidden, -np.inf, scale * (qq @ kk.T))
                none = hidden.all(1)
                m = np.where(none, 0.0, x.max(1, initial=-np.inf))
                p = np.where(hidden, 0.0, np.exp(x - m[:, None]))
                total = p.sum(1)
                # masked keys have no part: 0 * NaN must not reach a row
                pv = np.zeros((live, d))
                pa = np.zeros((live, d))
                clean = np.where(np.isfinite(vv), vv, 0.0)
                pv += p @ clean
                pa += p @ np.abs(clean)
                safe = np.where(none, 1.0, total)
                out[0][b, h, :live] = np.where(none[:, None], 0.0, pv / safe[:, None])
                out[1][b, h, :live] = np.where(none, -np.inf, m + np.log(safe))
                out[2][b, h, :live] = np.where(none[:, None], 0.0, pa / safe[:, None])
                sv = np.repeat(np.asarray(vscale, np.float64)[pages, hk], PAGE)[:n]
                out[4][b, h, :live] = (~hidden).sum(1) * (p * sv).max(1, initial=0.0) / safe
                mag = np.where(hidden, 0.0, scale * (np.abs(qq) @ np.abs(kk).T))
                out[3][b, h, :live] = np.nan_to_num(mag).max(1, initial=0.0)
    return out
