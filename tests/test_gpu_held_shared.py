"""Sequences that share the pages of a common beginning: their keys are weighed in a call for
each, and they are cut down apart in one call, into pages of their own."""
import math

import numpy as np
import pytest
import torch

from oracle import evict as E

from cache_common import PAGE, values
from gpu_common import need_gpu
from test_gpu_cache_evict import check as check_evict
from test_gpu_cache_fwd import make
from test_gpu_cache_weights import forward, host, ints


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 20])
def test_weights_in_a_call_for_each_sequence(N):
    fm = need_gpu()
    H, Hk, d, lens = 8, 2, 64, [300, 200, 131 + N]
    q, cache, table, gen = make(fm, 3, H, Hk, N, d, lens, seed=N)
    table[1, :2] = table[0, :2]
    table[2, :2] = table[0, :2]
    start = [0, 128, 128]  # the first counts for the shared keys from nothing, the others add
    lse = forward(fm, q, cache, table, lens, None, None)
    old = torch.rand((cache.k8.shape[0], Hk, PAGE), generator=gen).cuda()
    w, ws = old.clone(), fm.alloc_cache_weights_workspace(1, H, Hk, N, d, table.shape[1])
    for b in range(3):
        at = slice(b, b + 1)
        fm.flashmask_cache_weights(q[at], cache, table[at].contiguous(), ints(lens[at]), lse[at].contiguous(), w, ws,
                                   start=ints(start[at]))
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    want, bound = host(old).astype(np.float64), np.zeros(old.shape)
    for b in range(3):
        at = slice(b, b + 1)
        want, tol = E.weigh(q[at].double().cpu().numpy(), values(cache.k8), host(cache.kscale), host(table)[at], lens[at],
                            None, host(lse)[at], want, start[at], 1 / math.sqrt(d))
        bound += tol + np.abs(want) * 2.0 ** -24  # (each call's sums start from rounded ones)
    assert np.all(np.abs(host(w) - want) <= bound)


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["random", "ties"])
def test_eviction_apart(weights):
    fm = need_gpu()

    def edit(cache, table, gen):
        table[1, :3] = table[0, :3]
        table[2, :1] = table[0, :1]
    check_evict(fm, [700, 300, 65], [350, 120, 64], 2, 128, 4, 20, True, weights, edit=edit)
