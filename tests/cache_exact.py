"""Long attention cases whose sums are exact, so that a bound can be as tight as the
rounding of O and a page that is lost, or read from another's place, shows.

Scores are whole numbers of log2 units: a query row has one value q0 in {0, 1, 2}
throughout, a key one element that is not zero, s / kscale with s in {0, -1, -2, -3} and
kscale a power of two, and the call's scale is fp32's ln 2, which times fp32's log2(e)
rounds to 1. So P is a power of two between 2^-6 and 1. Values are +-1 or +-2 times a
power of two in {1/2, 1, 2}, the sign constant over a page's column: a page adds about 64
of a sign of its own to every column of O, where all pages together add the square root of
their number of that.

Every product and partial sum of a row is a multiple of its least P times 1/2, and below
2^24 of them (checked), hence exact in fp32, and P is exact in fp16. What
is left are the factors between references (the two running maxima take at most 15 values
in a warp, then at most three levels of joins and the last division: under 32 steps of
2^-22) and the rounding of O."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 64
SCALE = float(np.float32(math.log(2)))
assert np.float32(SCALE) * np.float32(1.4426950408889634) == np.float32(1)

# name: B, H, Hk, N, d, lengths, pages of the table, mask, mask heads
CASES = {
    # segments cut into parts, few rows and many
    "one_head_64": (1, 4, 1, 1, 64, [64 * 700], 701, None, 1),
    "two_lengths": (2, 4, 1, 1, 128, [64 * 230 + 5, 64 * 60], 240, None, 1),
    "sixteen_rows": (3, 6, 1, 3, 64, [30000, 100, 0], 470, None, 1),
    "rows_420": (1, 2, 1, 40, 64, [64 * 420], 420, None, 1),
    "rows_330": (1, 1, 1, 140, 128, [64 * 330 + 1], 340, None, 1),
    "rows_three": (3, 3, 1, 50, 128, [20000, 64 * 40, 9000], 330, None, 1),
    "one_row_40000": (1, 2, 1, 1, 64, [40000], 626, None, 1),
    "rows_40000": (1, 2, 1, 140, 64, [40000], 626, None, 1),
    # the line of many segments cut into equal runs
    "line": (40, 8, 4, 1, 64, [3000 - 61 * b for b in range(40)], 48, None, 1),
    "line_rows": (30, 4, 4, 70, 128, [4000 - 117 * b for b in range(30)], 64, None, 1),
    # page lists: every variant of the classification (tables of up to 32, 64, 128 pages by
    # one CTA, then by clusters of 2, 4 and 8; ranks without pages, several passes)
    "list_33": (2, 4, 2, 1, 64, [33 * 64, 1900], 33, "window", 2),
    "list_70": (2, 4, 2, 1, 64, [70 * 64 - 3, 4100], 70, "window", 1),
    "list_128": (1, 8, 2, 2, 128, [128 * 64], 128, "shares", 8),
    "list_129": (2, 2, 1, 40, 64, [129 * 64, 5000], 129, "window", 1),
    "list_161": (1, 4, 4, 1, 128, [161 * 64 - 33], 161, "last", 4),
    "list_290": (2, 4, 1, 3, 64, [290 * 64, 11111], 290, "shares", 2),
    "list_290_rows": (1, 2, 2, 150, 128, [290 * 64 - 1], 290, "upper", 2),
    "list_513": (2, 2, 2, 1, 64, [513 * 64, 20001], 513, "shares", 1),
    "list_513_rows": (1, 3, 1, 50, 64, [513 * 64 - 7], 513, "shares", 3),
    "list_1100": (1, 4, 2, 1, 64, [1100 * 64 - 9], 1100, "window", 2),
    "list_2048": (3, 2, 1, 1, 64, [2048 * 64, 70000, 333], 2048, "window", 2),
    "list_2048_rows": (1, 1, 1, 140, 64, [2048 * 64 - 100], 2048, "last", 1),
    "list_joined_twice": (1, 4, 1, 1, 64, [700 * 64], 700, "shares", 1),
    "list_joined_twice_rows": (1, 1, 1, 140, 64, [700 * 64], 700, "upper", 1),
    "list_line": (40, 8, 4, 1, 64, [4480 - 91 * b for b in range(40)], 70, "shares", 4),
    "list_line_rows": (30, 4, 4, 70, 64, [4400 - 117 * b for b in range(30)], 70, "window", 2),
    # long tables, short sequences
    "list_sparse": (6, 8, 2, 4, 64, [64 * 1500, 1, 0, 64, 129, 4000], 1500, "last", 8),
}


def mask_vectors(kind, B, Hm, L, lens):
    """lts, lte, uts, ute [B, Hm, L] (or None). window: a band and a prefix, wider with the
    mask head; shares: every third run of 37 pages (of each head another third) and the
    table's first eighth are hidden from all rows, and a few keys of every 11th page from
    all but the first rows; last: only keys of the last tenth are seen; upper: an
    interval above the diagonal's side ends inside pages."""
    j = np.arange(L, dtype=np.int64)
    h = np.arange(Hm, dtype=np.int64)[:, None]
    n = np.asarray(lens, np.int64)[:, None, None]
    far = 2 ** 31 - 1
    one = np.ones((B, Hm, L), np.int64)
    lts, lte, uts, ute = L * one, far * one, None, None
    if kind == "window":
        w = np.maximum(n // 2, 1500) + 37 * h
        lts = np.where(j < 100, far, j + w) * one
    elif kind == "shares":
        hide = ((j // (64 * 37)) % 3 == h % 3) & (j >= 64) | (j < L // 8) & (j >= 64)
        lts = np.where(hide, 0, far) * one
        uts = np.where((j // PAGE % 11 == 5) & (j % PAGE > 50), n - 2, 0) * one
        ute = np.where((j // PAGE % 11 == 5) & (j % PAGE > 50), far, 0) * one
    elif kind == "last":
        lts = np.where(j < 9 * n // 10 - 17 * h, 0, far) * one
    elif kind == "upper":
        lts = lte = None
        hide = (j // 29) % 4 == h % 4
        uts, ute = np.where(hide, n - 100, 0) * one, np.where(hide, n - 20, 0) * one
    return [None if x is None else torch.from_numpy(np.minimum(x, far).astype(np.int32))
            for x in (lts, lte, uts, ute)]


def build(name):
    """CPU tensors of a case: q, k8, kscale, v8, vscale, table, lens, mask vectors, causal."""
    B, H, Hk, N, d, lens, most, kind, Hm = CASES[name]
    gen = torch.Generator().manual_seed(sum(map(ord, name)))
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen)
    table = torch.full((B, most), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    pick = lambda shape, values: torch.tensor(values)[torch.randint(0, len(values), shape, generator=gen)]
    kscale = pick((pages, Hk), [0.25, 0.5, 1.0, 2.0, 4.0])
    vscale = pick((pages, Hk), [0.5, 1.0, 2.0])
    s = pick((pages, Hk, PAGE), [0.0, -1.0, -2.0, -3.0]) / kscale[..., None]
    where = torch.randint(0, d, (pages, Hk, PAGE, 1), generator=gen)
    k8 = torch.zeros((pages, Hk, PAGE, d)).scatter_(3, where, s[..., None])
    v8 = pick((pages, Hk, d, 1), [-1.0, 1.0]) * pick((pages, Hk, d, PAGE), [1.0, 2.0])
    f8 = lambda x: x.to(torch.float8_e4m3fn)
    assert torch.equal(f8(k8).float(), k8)
    q = pick((B, H, N, 1), [0.0, 1.0, 2.0]).expand(B, H, N, d).contiguous().bfloat16()
    vectors = [None] * 4 if kind is None else mask_vectors(kind, B, Hm, most * PAGE, lens)
    return q, f8(k8), kscale, f8(v8), vscale, table, lens, vectors


def tolerances(o, lse, pv):
    """Bounds of O and LSE from the oracle's O, LSE and sum P |V| / sum P: 32 steps of
    2^-22 for the factors, half a bf16 step (2^-8, with what the value's own error adds)
    for O, 2^-22 relative and 2^-20 for the logarithm and its product with ln 2."""
    return pv * 2.0 ** -17 + np.abs(o) * 2.0 ** -8 * 1.02, \
        2.0 ** -17 + 2.0 ** -20 + np.abs(np.where(np.isfinite(lse), lse, 0.0)) * 2.0 ** -22
