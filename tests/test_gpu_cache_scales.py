"""Scales of a cache that are no scales, and scales and queries whose product passes
fp32, against the fp64 definition."""
import math

import pytest
import torch

from cache_common import PAGE
from gpu_common import need_gpu
from test_gpu_cache_fwd import check, make, run

pytestmark = pytest.mark.gpu

NONE = [float("nan"), float("inf"), -float("inf"), -0.25]


@pytest.mark.parametrize("which", ["kscale", "vscale"])
@pytest.mark.parametrize("N", [1, 6, 140])
@pytest.mark.parametrize("d", [64, 128])
def test_a_page_without_a_scale(which, N, d):
    """Rows that see a key of the page get NaN, in its cache head only; rows from which
    causality, the mask or the length hides all of its keys are as they were."""
    fm = need_gpu()
    lens = [200, 333]
    q, cache, table, _ = make(fm, 2, 4, 2, N, d, lens, seed=3)
    L = table.shape[1] * PAGE
    page = int(table[0, 2])  # keys 128 .. 191 of sequence 0
    lts = torch.full((2, 1, L), L, dtype=torch.int32)
    lts[0, 0, 128:192] = 200 - N + N // 2  # hidden from the later half of the rows
    mask = fm.DeviceMask(lts.cuda(), torch.full_like(lts, L).cuda(), None, None, True)
    hidden = lts.clone()
    hidden[0, 0, 128:192] = 0
    never = fm.DeviceMask(hidden.cuda(), torch.full_like(lts, L).cuda(), None, None, True)
    scales = getattr(cache, which)
    good = scales[page, 1].item()
    for value in NONE:
        for m, rows in ((None, range(N)), (mask, range(N // 2)), (never, ())):
            scales[page, 1] = value
            o, lse = run(fm, q, cache, table, lens, mask=m)
            scales[page, 1] = good
            bad = {(0, h, t) for h in (2, 3) for t in rows if 200 - N + t >= 128}
            check(o, lse, q, cache, table, lens, mask=m, nan_rows=bad)


@pytest.mark.parametrize("N", [1, 6, 140])
def test_scales_of_zero(N):
    # zero times any code: scores of 0, values of 0; the sign of zero does not count
    fm = need_gpu()
    lens = [200, 333]
    q, cache, table, _ = make(fm, 2, 4, 2, N, 128, lens, seed=4)
    cache.kscale[int(table[0, 1])] = 0.0
    cache.kscale[int(table[0, 2])] = -0.0
    cache.vscale[int(table[1, 0])] = -0.0
    cache.vscale[table[0, :4].long()] = 0.0
    o, lse = run(fm, q, cache, table, lens)
    check(o, lse, q, cache, table, lens)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("N", [1, 6, 140])
@pytest.mark.parametrize("d", [64, 128])
def test_factors_that_pass_fp32(N, d):
    """Queries with an element of 2^26 and keys of scale 2^119, where the factor between
    a sum of codes and its score is above 2^128. Keys that are zero where the query is
    large have finite scores, and these count: all zero in sequence 0 (weights equal),
    one key of 2^110 in sequence 1 (it takes all the weight)."""
    fm = need_gpu()
    lens = [N + 300, N + 300]
    q, cache, table, _ = make(fm, 2, 4, 2, N, d, lens, seed=5)
    q[..., 0], q[..., 1], q[..., 2:] = 2.0 ** 26, 1.0, 0.0
    k8 = cache.k8.view(torch.uint8)
    k8[..., :2] = 0
    cache.kscale[:] = 2.0 ** 119
    page = int(table[1, 1])
    k8[page, :, 7, 1] = 1  # the smallest code, 2^-9: key 71 of sequence 1 scores 2^110 / sqrt(d)
    o, lse = run(fm, q, cache, table, lens)
    v = cache.v8.float() * cache.vscale[..., None, None]
    n = torch.arange(lens[0] - N, lens[0]) + 1  # keys that row t of sequence 0 sees
    assert torch.allclose(lse[0].cpu().double(), n.double().log().expand(4, N), rtol=0, atol=2.0 ** -18)
    assert torch.isfinite(o).all()
    want = v[page, :, :, 7].repeat_interleave(2, 0)[:, None].expand(4, N, d)
    assert torch.equal(o[1], want.bfloat16())
    assert torch.allclose(lse[1].cpu().double(), torch.tensor(2.0 ** 110 / math.sqrt(d)).double(), rtol=2.0 ** -20, atol=0)
    # sequence 0 as a mean, in fp64: P = 1 throughout, so only O's rounding is left
    pages = table[0, :-(-lens[0] // PAGE)].long()
    vals = v[pages].permute(1, 0, 3, 2).reshape(2, -1, d)[:, :lens[0]].double().cpu()
    mean = (vals.cumsum(1)[:, -N:] / n[:, None]).repeat_interleave(2, 0)
    err = (o[0].double().cpu() - mean).abs()
    assert (err <= mean.abs() * 2.0 ** -8 * 1.02 + vals.abs().amax() * 2.0 ** -16).all()
