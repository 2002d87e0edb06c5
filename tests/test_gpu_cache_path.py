"""Rotary positions, the cache and attention over it as a server uses them: a prompt
in chunks, then token by token, sequences of uneven length, under a column-wise mask.

Every step's attention is checked against the fp64 definition on the cache's codes;
the codes against the fp64 definition of the writes; and the whole prompt against the
library's own forward on the dequantised keys and values, which e4m3 codes times
powers of two make exact in bf16."""
import math

import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import workloads as W
from oracle import cache as C

from cache_common import PAGE, attention_bounds, cache_arrays
from gpu_common import TOL_LSE, TOL_O, need_gpu

pytestmark = pytest.mark.gpu


def dequantised(cache, table, b, n):
    pages = table[b, :-(-n // PAGE)].long()
    k = cache.k8[pages].float() * cache.kscale[pages][..., None, None]
    v = cache.v8[pages].float() * cache.vscale[pages][..., None, None]
    Hk, d = k.shape[1], k.shape[3]
    k = k.transpose(0, 1).reshape(Hk, -1, d)[:, :n]
    v = v.permute(1, 0, 3, 2).reshape(Hk, -1, d)[:, :n]
    assert torch.equal(k, k.bfloat16().float()) and torch.equal(v, v.bfloat16().float())
    return k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("masked", [False, True])
def test_prompt_in_chunks_then_tokens(d, masked):
    fm = need_gpu()
    B, H, Hk = 3, 8, 2
    total, chunk = [333, 70, 200], 128
    gen = torch.Generator().manual_seed(11)
    L = 6 * PAGE
    x = torch.randn((B, L, (H + 2 * Hk) * d), generator=gen).bfloat16().cuda()
    freqs, mscale = fm.rope_frequencies(d, 10000.0, "parts", 4.0, 128)
    order = torch.randperm(B * 6 + 3, generator=gen)[:B * 6].int()
    table = order.view(B, 6).cuda().contiguous()
    cache = fm.KVCache.empty(B * 6 + 3, Hk, d)
    ws = fm.alloc_cache_workspace(B, H, Hk, chunk, d, 6)
    j = torch.arange(L, dtype=torch.int32)
    lts = torch.where(j < 16, L, j + 90).int().expand(B, 1, L).contiguous().cuda()
    mask = fm.DeviceMask(lts, torch.full_like(lts, L), None, None, True) if masked else None
    vec = dict(lts=lts.cpu().numpy(), lte=np.full((B, 1, L), L)) if masked else {}
    held = [0] * B
    want = cache_arrays(cache)
    steps = [chunk] * 3 + [1] * 8
    f = lambda t: t.double().cpu().numpy()
    for N in steps:
        new = [min(N, t - h) if N > 1 else 1 for t, h in zip(total, held)]
        rows = torch.stack([x[b, h:h + N] if h + N <= L else
                            torch.cat([x[b, h:], x[b, :h + N - L]]) for b, h in enumerate(held)])
        q, k, v = (rows[..., a * d:e * d].unflatten(2, (e - a, d)).transpose(1, 2)
                   for a, e in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
        start = torch.tensor(held, dtype=torch.int32, device="cuda")
        count = torch.tensor(new, dtype=torch.int32, device="cuda")
        pos = (start[:, None] + torch.arange(N, device="cuda")).int().contiguous()
        q, k = fm.flashmask_rope(q, k, freqs, positions=pos, mscale=mscale)
        fm.flashmask_cache_append(cache, table, k, v, start, ws, count=count)
        o, lse = fm.flashmask_fwd_cache(q, cache, table, start + count, ws, mask=mask, q_lens=count)
        assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
        want = C.append(*want, table.cpu().numpy(), f(k), f(v), held, new)
        for got, ref in zip(cache_arrays(cache), want):
            assert np.array_equal(got, ref)
        held = [h + n for h, n in zip(held, new)]
        ref = C.attend(f(q), *want, table.cpu().numpy(), held, new, 1 / math.sqrt(d), **vec)
        tol_o, tol_l = attention_bounds(ref, max(held))
        for b, n in enumerate(new):
            assert np.all(np.abs(f(o)[b, :, :n] - ref[0][b, :, :n]) <= tol_o[b, :, :n])
            assert np.all(np.abs(f(lse)[b, :, :n] - ref[1][b, :, :n]) <= tol_l[b, :, :n])


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_at_once_equals_the_forward(d):
    # a prompt of two documents behind one another, in one call of N = length
    fm = need_gpu()
    B, H, n = 1, 4, 700
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((B, H, n, d), generator=gen).bfloat16().cuda() for _ in range(3))
    pages = -(-n // PAGE)
    cache = fm.KVCache.empty(pages, H, d)
    table = torch.randperm(pages, generator=gen).int().view(1, pages).cuda()
    ws = fm.alloc_cache_workspace(B, H, H, n, d, pages)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    fm.flashmask_cache_append(cache, table, k, v, zero, ws)
    spec = W.document_bounds(1, 1, [300, 400])
    m = fm.DeviceMask.from_spec(spec)
    pad = lambda t: torch.nn.functional.pad(t, (0, pages * PAGE - n)).contiguous()
    o, lse = fm.flashmask_fwd_cache(q, cache, table, zero + n, ws,
                                    mask=fm.DeviceMask(pad(m.lts), pad(m.lte), None, None, spec.causal))
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    kd, vd = dequantised(cache, table, 0, n)
    fws = fm.alloc_workspace(B, H, 1, n, d, for_bwd=False)
    o2, lse2 = fm.flashmask_fwd(q, kd[None].contiguous(), vd[None].contiguous(), m, fws)
    assert (o.float() - o2.float()).abs().max() <= 2 * TOL_O
    assert (lse - lse2).abs().max() <= 2 * TOL_LSE
