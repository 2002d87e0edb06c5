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


def attention_bounds(ref, keys):
    """Elementwise error bounds of O and LSE from the oracle's (O, LSE, PV, smag, top)
    for at most `keys` keys.

    delta bounds the error of a score: the products of fp16 query and codes are exact,
    their fp32 sums lose up to 2^-22 of the largest term in each of at most 8 steps
    (2^-19 of sum |q k|), and the exponent 2^-22 of the score. P carries 2 delta +
    2^-20 (the exponential's error) relative and 2^-11 for its rounding to fp16; below
    fp16's normal range half a step is 2^-32 of the row's largest P_j times value scale
    or less (2^-25 of a P stored as 2^7 P or more), for each key, times a code of at
    most 448. Sums over the keys add in chains of at most keys / 4 terms (l) or keys /
    16 instructions (O), each a step of 2^-23: keys * 2^-25 covers either. O is rounded
    to bf16 (2^-8)."""
    o, lse, pv, smag, top = ref
    delta = smag * 2.0 ** -18 + 2.0 ** -20
    sums = keys * 2.0 ** -25
    tol_o = pv * (2.0 ** -11 + 2.0 ** -19 + 2 * sums + 2 * delta[..., None]) + \
        top[..., None] * 448 * 2.0 ** -32 * keys + np.abs(o) * 2.0 ** -8 * 1.02 + 1e-30
    tol_lse = delta + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -22 + 2.0 ** -20 + sums
    return tol_o, tol_lse
