"""Scores so large that the scale of V would be lost beside them: O is the mean of the
two keys that share a row's largest score, whatever its size."""
import math

import pytest
import torch

from cache_common import PAGE, cache_arrays
from gpu_common import need_gpu
from test_gpu_cache_fwd import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mag", [2.0 ** 7, 2.0 ** 14, 2.0 ** 20, 2.0 ** 31, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("H,N,lens", [
    (4, 1, [300, 64 * 90, 40]), (4, 6, [300, 64 * 90, 70]), (2, 140, [400, 64 * 90, 150]),
    (2, 1, [64 * 420]), (2, 40, [64 * 420]), (1, 1, [64 * 40] * 160)])
def test_two_keys_share_the_weight(mag, H, N, lens):
    fm = need_gpu()
    B, Hk, d = len(lens), 1, 64
    q, cache, table, gen = make(fm, B, H, Hk, N, d, lens, seed=11)
    q[..., 0], q[..., 1:] = mag, 0.0
    # dimension 0 of K: 0 or 1, and 4 at two keys that every row sees; scores of 4 mag / 8
    # against at most mag / 8, so the others weigh e^-48 or less of the two
    code = torch.randint(0, 2, cache.k8.shape[:3], generator=gen).float()
    cache.kscale[:] = 1.0
    cache.vscale.copy_(torch.exp2(torch.rand(cache.vscale.shape, generator=gen) * 20 - 10))
    t, picks = table.cpu(), []
    for b, n in enumerate(lens):
        pick = torch.randperm(n - N + 1, generator=gen)[:2].tolist()
        picks.append(pick)
        for j in pick:
            code[t[b, j // PAGE], 0, j % PAGE] = 4.0
    cache.k8[..., 0] = code.cuda().to(torch.float8_e4m3fn)
    o, lse = run(fm, q, cache, table, lens)
    _, _, v8, vs = cache_arrays(cache)
    for b, pick in enumerate(picks):
        v = torch.stack([torch.from_numpy(v8[p, 0, :, j % PAGE] * vs[p, 0])
                         for j in pick for p in [int(t[b, j // PAGE])]])
        want = v.sum(0) / len(pick)
        # P is rounded to fp16 and O to bf16; 2^-20 for the factors between pages and
        # states; the other keys' part, e^-48 each of values up to 448 * 2^10
        others = lens[b] * math.exp(-3 * mag / 8) * 448 * 2.0 ** 10
        tol = v.abs().sum(0) / len(pick) * (2.0 ** -11 + 2.0 ** -17) + want.abs() * 2.0 ** -8 * 1.02 + others
        assert (o[b].double().cpu() - want).abs().le(tol).all(), (b, pick)
        top = mag / 2 + math.log(len(pick))
        assert (lse[b].double().cpu() - top).abs().max() <= top * 2.0 ** -20 + 2.0 ** -18 + lens[b] * math.exp(-3 * mag / 8)
