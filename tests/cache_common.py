"""Shared helpers of the rotary and paged-cache tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import fp8 as F

TABLE = F.e4m3_table()
PAGE = 64


def values(codes: torch.Tensor) -> np.ndarray:
    """fp64 values of e4m3 codes (NaN for the NaN codes)."""
    return TABLE[codes.contiguous().view(torch.uint8).cpu().numpy()]


def random_cache(fm, pages, Hk, d, gen, spread=3, device="cuda"):
    """A cache whose pages hold normal values at scales that differ by page."""
    c = fm.KVCache.empty(pages, Hk, d, device=device)
    for t in (c.k8, c.v8):
        t.copy_((torch.randn(t.shape, generator=gen) * 96).clamp(-448, 448).to(torch.float8_e4m3fn))
    for t in (c.kscale, c.vscale):
        t.copy_(torch.exp2(torch.randint(-7 - spread, -6, t.shape, generator=gen).float()))
    return c


def random_table(lens, max_pages, gen, pages=None, device="cuda"):
    """int32 [B, max_pages] with distinct pages in random order; entries that no
    token needs are out of range (they must not be read)."""
    need = [-(-int(n) // PAGE) for n in lens]
    pages = sum(need) if pages is None else pages
    order = torch.randperm(pages, generator=gen)
    t = torch.full((len(need), max_pages), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n].int()
        at += n
    return t.to(device)


def cache_arrays(c):
    return (values(c.k8), c.kscale.double().cpu().numpy(), values(c.v8),
            c.vscale.double().cpu().numpy())


def attention_bounds(ref):
    """Elementwise error bounds of O and LSE from the oracle's (O, LSE, PV, smag, top).

    delta bounds the error of a score: fp32 sums of d products in the tensor
    cores (alignment to the largest loses up to 2^-22 of it a step, at most 8
    steps of 32: 2^-19 of sum |q k|), the query as two or more parts of 4 bits
    (2^-22 of its largest), and 2^-22 of the score in the exponent. P carries
    2 delta + 2^-20 (the exponential's error) relative and 2^-8 for its own
    rounding to two parts of 4 bits; parts below the smallest step lose up to
    2^-22 of the row's largest P_j times value scale for each key (times a code
    of at most 448). O is rounded to bf16 (2^-8)."""
    o, lse, pv, smag, top = ref
    delta = smag * 2.0 ** -18 + 2.0 ** -20
    tol_o = pv * (2.0 ** -8 + 2 * delta[..., None]) + top[..., None] * 448 * 2.0 ** -22 + np.abs(o) * 2.0 ** -8 * 1.02 + 1e-30
    tol_lse = delta + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -22 + 2.0 ** -20
    return tol_o, tol_lse
