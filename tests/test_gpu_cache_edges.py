"""The largest and oddest calls that the header allows: the longest table, the most
sequences and heads, query heads that fill several tiles, more query rows than keys,
counts out of range, calls side by side, and a first call inside a capture."""
import math
import os
import subprocess
import sys

import pytest
import torch

from cache_common import PAGE, random_cache
from cache_exact import SCALE
from gpu_common import need_gpu
from test_gpu_cache_fwd import MARK, check, make, mask_of, run

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def attend64(q, cache, table, lens, q_lens, scale, mask=None):
    """O, LSE, sum P |V| / sum P and the scores' magnitude in fp64 on the GPU, one batch."""
    B, H, N, d = q.shape
    Hk = cache.k8.shape[1]
    t = table.long().clamp(0, cache.k8.shape[0] - 1)
    M = t.shape[1]
    f = lambda x: x.view(torch.uint8)[t].view(torch.float8_e4m3fn).double()
    k = (f(cache.k8) * cache.kscale[t].double()[..., None, None]).transpose(1, 2).reshape(B, Hk, M * PAGE, d)
    v = (f(cache.v8) * cache.vscale[t].double()[..., None, None]).permute(0, 2, 1, 4, 3).reshape(B, Hk, M * PAGE, d)
    live = torch.full_like(lens, N) if q_lens is None else q_lens
    i = ((lens - live)[:, None] + torch.arange(N, device=q.device))[:, None, :, None]
    j = torch.arange(M * PAGE, device=q.device)
    hidden = (j > i) | (j >= lens[:, None, None, None])
    if mask is not None:
        hidden = hidden | ((mask.lts[:, :, None] <= i) & (i < mask.lte[:, :, None]))
    hidden = hidden.repeat_interleave(H // hidden.shape[1], 1) if hidden.shape[1] > 1 else hidden
    qd = q.double().view(B, Hk, H // Hk * N, d)
    x = (scale * (qd @ k.transpose(-1, -2))).view(B, H, N, -1).masked_fill(hidden, -math.inf)
    size = (scale * (qd.abs() @ k.abs().transpose(-1, -2))).view(B, H, N, -1).masked_fill(hidden, 0.0).amax(-1)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse.clamp(min=-1e300)[..., None]).view(B, Hk, H // Hk * N, -1)
    return (p @ v).view(B, H, N, d), lse, (p @ v.abs()).view(B, H, N, d), size


def close(o, lse, ref, keys):
    """The bounds of cache_common.attention_bounds for few keys and V scales within 2^6."""
    want, wl, pv, size = ref
    none = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse), none) and (o[none] == 0).all()
    delta = size * 2.0 ** -18 + 2.0 ** -20
    tol = pv * (2.0 ** -11 + 2.0 ** -19 + keys * 2.0 ** -24 + 2 * delta[..., None]) + want.abs() * 2.0 ** -8 * 1.02 + \
        pv.amax(-1, keepdim=True) * 2.0 ** -16
    assert ((o.double() - want).abs() <= tol).all()
    tl = delta + wl.abs() * 2.0 ** -22 + 2.0 ** -20 + keys * 2.0 ** -25
    assert ((lse.double() - wl).abs() <= tl)[~none].all()


@pytest.mark.parametrize("N", [1, 140])
@pytest.mark.parametrize("masked", [False, True])
def test_the_longest_table(N, masked):
    # 2^21 tokens; sums exact but for their last joins, as in cache_exact
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(N)
    M, d = (1 << 21) // PAGE, 64
    pick = lambda shape, values: torch.tensor(values, device="cuda")[
        torch.randint(0, len(values), shape, generator=gen, device="cuda")]
    cache = fm.KVCache.empty(M, 1, d)
    cache.vscale.copy_(pick((M, 1), [0.5, 1.0, 2.0]))
    s = pick((M, 1, PAGE), [0.0, -1.0, -2.0, -3.0])
    k = torch.zeros((M, 1, PAGE, d), device="cuda")
    k.scatter_(3, torch.randint(0, d, (M, 1, PAGE, 1), generator=gen, device="cuda"), s[..., None])
    cache.k8.copy_(k.to(torch.float8_e4m3fn))
    cache.v8.copy_((pick((M, 1, d, 1), [-1.0, 1.0]) * pick((M, 1, d, PAGE), [1.0, 2.0])).to(torch.float8_e4m3fn))
    table = torch.randperm(M, generator=gen, device="cuda").int()[None].contiguous()
    q0 = pick((1, 1, N, 1), [0.0, 1.0, 2.0])
    q = q0.expand(1, 1, N, d).bfloat16().contiguous()
    lens = torch.tensor([M * PAGE], dtype=torch.int32, device="cuda")
    mask = None
    if masked:  # the first third and every fifth run of 1000 keys are hidden
        j = torch.arange(M * PAGE, device="cuda")
        hide = (j < M * PAGE // 3) | (j // 1000 % 5 == 2)
        lts = torch.where(hide, 0, 2 ** 31 - 1).int()[None, None].contiguous()
        mask = fm.DeviceMask(lts, torch.full_like(lts, 2 ** 31 - 1), None, None, True)
    ws = fm.alloc_cache_workspace(1, 1, 1, N, d, M)
    o, lse = fm.flashmask_fwd_cache(q, cache, table, lens, ws, mask=mask, scale=SCALE)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    t = table[0].long()
    for row in sorted({0, N // 2, N - 1}):
        p = torch.exp2(s[t, 0].double() * q0[0, 0, row].double()).view(-1)
        p[M * PAGE - N + row + 1:] = 0.0
        if masked:
            p[hide] = 0.0
        v = cache.v8[t, 0].double() * cache.vscale[t, 0].double()[:, None, None]
        l = p.sum()
        want = torch.einsum("pk,pdk->d", p.view(M, PAGE), v) / l
        pv = torch.einsum("pk,pdk->d", p.view(M, PAGE), v.abs()) / l
        assert ((o[0, 0, row].double() - want).abs() <= pv * 2.0 ** -17 + want.abs() * 2.0 ** -8 * 1.02).all()
        assert (lse[0, 0, row].double() - l.log()).abs() <= 2.0 ** -17 + 2.0 ** -20 + l.log() * 2.0 ** -22


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,H,N", [(65535, 1, 1), (40000, 2, 9)])
def test_the_most_sequences(B, H, N, masked):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(B)
    cache = random_cache(fm, B, 1, 64, gen)
    table = torch.randperm(B, generator=gen).int()[:, None].contiguous().cuda()
    lens = torch.randint(0, PAGE + 1, (B,), generator=gen).int().cuda()
    q = torch.randn((B, H, N, 64), generator=gen).bfloat16().cuda()
    mask = None
    if masked:
        lts = (torch.arange(PAGE) + 20).int().expand(B, 1, PAGE).contiguous().cuda()
        mask = fm.DeviceMask(lts, torch.full_like(lts, 1000), None, None, True)
    ws = fm.alloc_cache_workspace(B, H, 1, N, 64, 1)
    o, lse = fm.flashmask_fwd_cache(q, cache, table, lens, ws, mask=mask)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for at in range(0, B, 8192):
        x = slice(at, min(B, at + 8192))
        m = None if mask is None else fm.DeviceMask(mask.lts[x], mask.lte[x], None, None, True)
        close(o[x], lse[x], attend64(q[x], cache, table[x], lens[x], None, 1 / 8, m), PAGE)


@pytest.mark.parametrize("H,Hk,N", [(65535, 65535, 1), (60000, 15000, 3)])
def test_the_most_heads(H, Hk, N):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(Hk)
    cache = random_cache(fm, 2, Hk, 64, gen)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    # the last tokens are written by the call before, page 0's scales grow
    k, v = (torch.randn((1, Hk, N, 64), generator=gen).bfloat16().cuda() for _ in range(2))
    ws = fm.alloc_cache_workspace(1, H, Hk, N, 64, 2)
    held = torch.tensor([100], dtype=torch.int32, device="cuda")
    fm.flashmask_cache_append(cache, table, k, v, held, ws)
    q = torch.randn((1, H, N, 64), generator=gen).bfloat16().cuda()
    lens = held + N
    o, lse = fm.flashmask_fwd_cache(q, cache, table, lens, ws)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    G, step = H // Hk, 3000
    for at in range(0, Hk, step):
        x, y = slice(at, min(Hk, at + step)), slice(at * G, min(Hk, at + step) * G)
        part = fm.KVCache(*(t[:, x].contiguous() for t in cache.tensors))
        close(o[:, y], lse[:, y], attend64(q[:, y], part, table, lens, None, 1 / 8), 100 + N)


@pytest.mark.parametrize("H,Hk,N,d,kind", [(300, 1, 1, 64, None), (129, 1, 2, 128, "random_head"),
                                           (256, 2, 1, 128, "random_kv"), (66, 2, 1, 64, "random_head")])
def test_heads_that_fill_tiles(H, Hk, N, d, kind):
    fm = need_gpu()
    lens = [500, 70, 0]
    q, cache, table, gen = make(fm, 3, H, Hk, N, d, lens, seed=H)
    mask = None if kind is None else mask_of(kind, 3, H, Hk, N, table.shape[1] * PAGE, gen, fm)
    o, lse = run(fm, q, cache, table, lens, None, mask)
    check(o, lse, q, cache, table, lens, None, mask)


def test_more_rows_than_keys():
    fm = need_gpu()
    N, lens = 70000, torch.tensor([300], dtype=torch.int32, device="cuda")
    q, cache, table, _ = make(fm, 1, 2, 1, N, 64, [300], seed=1)
    ws = fm.alloc_cache_workspace(1, 2, 1, N, 64, table.shape[1])
    o, lse = fm.flashmask_fwd_cache(q, cache, table, lens, ws)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    assert (o[:, :, :N - 300] == 0).all() and torch.isneginf(lse[:, :, :N - 300]).all()
    ref = attend64(q[:, :, N - 300:].contiguous(), cache, table, lens, None, 1 / 8)
    close(o[:, :, N - 300:], lse[:, :, N - 300:], ref, 300)


@pytest.mark.parametrize("N", [3, 50])
def test_counts_out_of_range_are_clamped(N):
    fm = need_gpu()
    lens = [200, 200, 200, 200]
    q, cache, table, gen = make(fm, 4, 4, 2, N, 64, lens, seed=N)
    wild, tame = [N + 7, -1, 2 ** 31 - 1, -2 ** 31], [N, 0, N, 0]
    for mask in (None, mask_of("window", 4, 4, 2, N, table.shape[1] * PAGE, gen, fm)):
        o, lse = run(fm, q, cache, table, lens, wild, mask)
        check(o, lse, q, cache, table, lens, tame, mask)
        assert (o[1] == MARK).all() and (lse[3] == MARK).all()
    k = torch.randn((4, 2, N, 64), generator=gen).bfloat16().cuda()
    other = fm.KVCache(*(t.clone() for t in cache.tensors))
    ws = fm.alloc_cache_workspace(4, 4, 2, N, 64, table.shape[1])
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for c, count in ((cache, wild), (other, tame)):
        fm.flashmask_cache_append(c, table, k, k, dev([100] * 4), ws, count=dev(count))
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for a, b in zip(cache.tensors, other.tensors):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_calls_side_by_side():
    # two streams, each with its workspace and graph, on one cache; and two graphs that
    # share a workspace, one after the other
    fm = need_gpu()
    sets = []
    for i, (H, N, lens) in enumerate([(8, 1, [9000, 64 * 90, 40]), (8, 40, [5000, 1200, 64 * 80])]):
        q, cache, table, gen = make(fm, 3, H, 2, N, 128, lens, seed=i)
        mask = mask_of("window_prefix", 3, H, 2, N, table.shape[1] * PAGE, gen, fm) if i else None
        ws = fm.alloc_cache_workspace(3, H, 2, 40, 128, 160)
        args = (q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        want = fm.flashmask_fwd_cache(*args, ws, mask=mask)
        sets.append((args, mask, ws, [t.clone() for t in want], torch.cuda.Stream()))
    torch.cuda.synchronize()

    def capture(i, ws):
        args, mask, _, _, _ = sets[i]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fm.flashmask_fwd_cache(*args, ws, mask=mask)
        return g, out

    graphs = [capture(i, sets[i][2]) for i in range(2)]
    for _ in range(20):
        for (g, _), s in zip(graphs, sets):
            with torch.cuda.stream(s[4]):
                g.replay()
    torch.cuda.synchronize()
    shared = [capture(i, sets[0][2]) for i in range(2)]
    for _ in range(10):
        for g, _ in shared:
            g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for _, out in (graphs[i], shared[i]):
            assert all(torch.equal(a, b) for a, b in zip(out, sets[i][3]))
        assert fm.flashmask_check_status(sets[i][2]) == (fm.FM_OK, 0)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from mask_aware_exact_gb300 import flashmask as fm
H, N, masked = {H}, {N}, {masked}
cache = fm.KVCache.empty(9, 2, 64)
table = torch.arange(9, dtype=torch.int32, device="cuda")[None]
q = torch.randn((1, H, N, 64), device="cuda").bfloat16()
k = torch.randn((1, 2, N, 64), device="cuda").bfloat16()
held = torch.tensor([300], dtype=torch.int32, device="cuda")
ws = fm.alloc_cache_workspace(1, H, 2, N, 64, 9)
freqs, _ = fm.rope_frequencies(64)
lts = torch.arange(9 * 64, dtype=torch.int32, device="cuda")[None, None] + 50
mask = fm.DeviceMask(lts.contiguous(), torch.full_like(lts, 9999), None, None, True) if masked else None

def step():
    q2, k2 = fm.flashmask_rope(q, k, freqs)
    fm.flashmask_cache_append(cache, table, k2, k, held, ws)
    return fm.flashmask_fwd_cache(q2, cache, table, held + N, ws, mask=mask)

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
"""


@pytest.mark.parametrize("H,N,masked", [(8, 1, False), (8, 4, True), (8, 40, False), (8, 40, True)])
def test_the_first_call_of_a_process_is_captured(H, N, masked):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, H=H, N=N, masked=masked)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
