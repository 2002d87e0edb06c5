"""Gradients of the normed rotary positions where the sums over a head would pass fp32.
The tolerance is test_gpu_norm_rope's: scaling by powers of two adds no rounding."""
import numpy as np
import pytest
import torch

from oracle import norm as O

from gpu_common import need_gpu
from test_gpu_norm_rope import check_backward, f64

# size of x and of its output's gradient: the sum of g w x alone past fp32, both sums, neither
# (beside them), gradients near fp32's largest
SIZES = [(1e18, 1e20), (1e19, 3e36), (30.0, 1e37), (1e30, 1e30), (3e37, 1e-20), (3e37, 1e36), (1.0, 1.0), (1e-8, 1e-8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (33, 20), (256, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_and_gradients_of_any_size(interleaved, d, rot, dtype):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(d)
    n = len(SIZES)
    a, z = (torch.tensor([s[i] for s in SIZES], dtype=torch.float64)[None, None, :, None] for i in (0, 1))
    rn = lambda: torch.randn((1, 3, n, d), generator=gen, dtype=torch.float64).clamp(-4, 4)
    x, g = (rn() * a).to(dtype).cuda(), (rn() * z).to(dtype).cuda()
    w = (torch.rand(d, generator=gen) + 0.5).cuda()
    freqs, _ = fm.rope_frequencies(rot)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    ws = fm.alloc_norm_workspace(d)
    how = dict(interleaved=interleaved)
    for t in range(n):  # each size alone, for its weights' gradient too
        one = lambda v: v[:, :, t:t + 1]
        got = fm.flashmask_norm_rope_bwd(one(g), None, one(x), None, w, None, freqs, ws,
                                         positions=pos[:, t:t + 1].contiguous(), **how)
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all(), SIZES[t]
        check_backward(got[0], got[2], one(g), one(x), w, pos[:, t:t + 1], freqs, interleaved, 1.0, 1e-6)
    # side by side they do not touch one another
    both = fm.flashmask_norm_rope_bwd(g, None, x, None, w, None, freqs, ws, **how)
    want, _ = O.backward(f64(g), f64(x), f64(w), f64(pos), f64(freqs), interleaved)
    for t in range(n):
        one = lambda v: v[:, :, t:t + 1]
        alone = fm.flashmask_norm_rope_bwd(one(g), None, one(x), None, w, None, freqs, ws,
                                           positions=pos[:, t:t + 1].contiguous(), **how)
        assert torch.equal(one(both[0]), alone[0])
    assert np.isfinite(want).all()
