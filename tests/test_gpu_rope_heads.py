"""Rotary calls whose threads walk over several heads: every head has to come out as
it does in a call of its own (where each thread has one head), to the bit, in place
too; a few heads are compared with the fp64 definition."""
import pytest
import torch

from gpu_common import need_gpu
from test_gpu_rope import check

pytestmark = pytest.mark.gpu


# Heads of a thread: H * ceil(B * N * chunks / 256) / (4 * SMs), at most 16, where a token
# has d / 16 chunks in 16-bit types, d / 8 in fp32, and about d / 2 where elements are
# accessed one by one; on 152 SMs 2, 5, 8, 16 and 4, 8, 16.
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,dtype,odd", [
    (2, 13, 3, 1300, 128, 128, torch.bfloat16, False), (1, 33, 8, 2500, 128, 64, torch.float16, False),
    (3, 40, 5, 1277, 128, 128, torch.bfloat16, False), (1, 61, 19, 3920, 64, 64, torch.float32, False),
    (1, 17, 2, 512, 128, 118, torch.bfloat16, False), (2, 30, 8, 257, 128, 128, torch.bfloat16, True),
    (1, 70, 13, 500, 128, 44, torch.float16, False)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_of_a_thread(B, Hq, Hk, N, d, rot, dtype, odd, interleaved):
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(N)

    def tensor(H):
        x = torch.randn((B, H, N, d + 1 if odd else d), generator=gen, device="cuda").to(dtype)
        return x[..., 1:] if odd else x

    q, k = tensor(Hq), tensor(Hk)
    freqs, _ = fm.rope_frequencies(rot)
    pos = torch.randint(-(1 << 20), 1 << 20, (B, N), generator=gen, device="cuda", dtype=torch.int32)
    kw = dict(positions=pos, interleaved=interleaved, mscale=1.25)
    yq, yk = fm.flashmask_rope(q, k, freqs, **kw)
    for x, y in ((q, yq), (k, yk)):
        H = x.shape[1]
        for h in range(H):
            one, _ = fm.flashmask_rope(x[:, h:h + 1], None, freqs, **kw)
            assert torch.equal(one, y[:, h:h + 1]), h
        some = sorted({0, 1, H // 2, H - 1})
        check(y[:, some, ::7], x[:, some, ::7], pos[:, ::7], freqs, interleaved, 1.25, False, dtype)
    fm.flashmask_rope(q, k, freqs, out=(q, k), **kw)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    back = fm.flashmask_rope_bwd(q, k, freqs, **kw)
    for g, y in zip(back, (yq, yk)):
        some = sorted({0, g.shape[1] - 1})
        check(g[:, some, ::7], y[:, some, ::7], pos[:, ::7], freqs, interleaved, 1.25, True, dtype)
