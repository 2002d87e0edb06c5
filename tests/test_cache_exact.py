"""The cases of cache_exact keep what their bounds assume, and the bounds reject what
they are for: a page of V lost, a page lost altogether, a page's V read from its
neighbour. Needs no GPU."""
import numpy as np
import pytest
import torch

from cache_common import TABLE
from cache_exact import CASES, PAGE, build, tolerances


def values(codes):
    return TABLE[codes.contiguous().view(torch.uint8).numpy()]


@pytest.mark.parametrize("name", list(CASES))
def test_bounds_reject_a_lost_page(name):
    B, H, Hk, N, d, lens, most, kind, Hm = CASES[name]
    q, k8, kscale, v8, vscale, table, lens, vectors = build(name)
    lts, lte, uts, ute = (None if t is None else t.numpy() for t in vectors)
    pairs = [(b, h) for b in range(B) if lens[b] for h in range(0, H, max(1, H // Hk))]
    seen = 0
    for b, h in pairs[:6]:
        n, hk = lens[b], h // (H // Hk)
        pages = table[b, :-(-n // PAGE)].long()
        rows = range(max(0, N - 4), N)  # the last rows
        i = np.array([n - N + t for t in rows])[:, None]
        j = np.arange(len(pages) * PAGE)[None]
        hidden = (j > i) | (j >= n)
        hm = h // (H // Hm)
        for lo, hi in ((lts, lte), (uts, ute)):
            if lo is not None:
                m = len(pages) * PAGE
                hidden = hidden | (lo[b, hm, :m] <= i) & (i < hi[b, hm, :m])
        k = (values(k8[pages, hk]) * kscale[pages, hk].numpy()[:, None, None]).reshape(-1, d)
        v = (values(v8[pages, hk]) * vscale[pages, hk].numpy()[:, None, None]).transpose(0, 2, 1)
        qq = q[b, h, list(rows)].double().numpy()
        s = qq @ k.T
        assert np.array_equal(s, np.round(s)) and s.max() <= 0 and s.min() >= -6
        p = np.where(hidden, 0.0, 2.0 ** s)
        part = np.einsum("tpk,pkd->tpd", p.reshape(len(rows), -1, PAGE), v)
        size = np.einsum("tpk,pkd->td", p.reshape(len(rows), -1, PAGE), np.abs(v))
        lp = p.reshape(len(rows), -1, PAGE).sum(2)
        l, acc = lp.sum(1), part.sum(1)
        live = l > 0
        if not live.any():
            continue
        part, size, lp, l, acc = part[live], size[live], lp[live], l[live], acc[live]
        unit = 2.0 ** s[live].min(1)
        assert (size.max(1) < 2 ** 24 * unit / 2).all() and (l < 2 ** 24 * unit).all()
        o, lse = acc / l[:, None], np.log(l)
        tol_o, tol_l = tolerances(o, lse, size / l[:, None])
        # every page that some of these rows see by more than a few keys
        for x in np.nonzero((lp >= 8 * lp.max() / PAGE).any(0))[0]:
            seen += 1
            lost = (acc - part[:, x]) / l[:, None]
            assert (np.abs(lost - o) > tol_o).any(), (b, h, x)
            with np.errstate(divide="ignore"):
                less = np.log(l - lp[:, x])
            both = np.divide(acc - part[:, x], (l - lp[:, x])[:, None], where=(l > lp[:, x])[:, None], out=np.zeros_like(acc))
            assert (np.abs(both - o) > tol_o).any() or (np.abs(less - lse) > tol_l).any(), (b, h, x)
            y = x + 1 if x + 1 < len(pages) else x - 1
            if y >= 0:
                other = np.einsum("tk,kd->td", p[live][:, PAGE * x:PAGE * x + PAGE], v[y])
                assert (np.abs((acc - part[:, x] + other) / l[:, None] - o) > tol_o).any(), (b, h, x, y)
    assert seen > 3
