"""The largest and oddest calls that the header allows of the normed positions, the weights
of cached keys and eviction: the longest table, the most sequences and heads, tensors past
2^31 elements, more query rows than keys, counts out of range, and a first call inside a
capture."""
import math
import os
import subprocess
import sys

import pytest
import torch

from cache_common import PAGE, random_cache
from gpu_common import need_gpu
from test_gpu_cache_fwd import make, mask_of
from test_gpu_cache_weights import check, forward, ints
from test_gpu_norm_rope import check_backward, check_forward, f64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def weigh64(q, cache, table, lens, lse, old, start, scale, lts=None):
    """Weights of the tables' pages [B, Hk, M * 64] in fp64 on the GPU and their bounds, those of
    oracle.evict.weigh; all rows of q are real, the mask is causal with lte past all."""
    B, H, N, d = q.shape
    Hk, M = cache.k8.shape[1], table.shape[1]
    t = table.long()
    k = cache.k8.view(torch.uint8)[t].view(torch.float8_e4m3fn).double() * cache.kscale[t].double()[..., None, None]
    k = k.transpose(1, 2).reshape(B, Hk, M * PAGE, d)
    i = (lens[:, None] - N + torch.arange(N, device=q.device))[:, None, :, None]
    j = torch.arange(M * PAGE, device=q.device)
    hidden = (j > i) | (j >= lens[:, None, None, None])
    if lts is not None:
        hidden = hidden | (lts[:, :, None] <= i)
    G = H // Hk
    qd = q.double().view(B, Hk, G * N, d)
    l = lse.double()[..., None]
    x = (scale * (qd @ k.transpose(-1, -2))).view(B, H, N, -1)
    size = (scale * (qd.abs() @ k.abs().transpose(-1, -2))).view(B, H, N, -1)
    p = torch.exp(x - l).masked_fill(hidden | torch.isneginf(l), 0.0)
    err = 2 * (size * 2.0 ** -18 + 2.0 ** -20) + l.clamp(min=-1e30).abs() * 2.0 ** -21 + 2.0 ** -19 + N * G * 2.0 ** -24
    got = p.view(B, Hk, G * N, -1).sum(2)
    tol = (p * err.masked_fill(torch.isneginf(l), 0.0)).view(B, Hk, G * N, -1).sum(2) + N * G * 2e-38
    was = old[t].double().transpose(1, 2).reshape(B, Hk, -1)
    had = torch.where(j < start[:, None, None], was, 0.0)
    want = torch.where(j < lens[:, None, None], had + got, was)
    return want, torch.where(j < lens[:, None, None], tol + (had.abs() + got) * 2.0 ** -23, 0.0)


def logsums(q, cache, table, lens, scale, lts=None):
    """LSE of the same rows, as fp32."""
    fm = need_gpu()
    B, H, N, d = q.shape
    ws = fm.alloc_cache_workspace(B, H, cache.k8.shape[1], N, d, table.shape[1])
    mask = None if lts is None else fm.DeviceMask(lts, torch.full_like(lts, 2 ** 31 - 1), None, None, True)
    return fm.flashmask_fwd_cache(q, cache, table, lens, ws, mask=mask, scale=scale)[1]


def weigh(q, cache, table, lens, lse, old, scale=None, start=None, lts=None):
    fm = need_gpu()
    B, H, N, d = q.shape
    ws = fm.alloc_cache_weights_workspace(B, H, cache.k8.shape[1], N, d, table.shape[1])
    mask = None if lts is None else fm.DeviceMask(lts, torch.full_like(lts, 2 ** 31 - 1), None, None, True)
    w = fm.flashmask_cache_weights(q, cache, table, lens, lse, old.clone(), ws, mask=mask, start=start, scale=scale)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    return w


def compare(w, table, want, tol):
    B, Hk, _ = want.shape
    got = w[table.long()].double().transpose(1, 2).reshape(B, Hk, -1)
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("N", [1, 40])
@pytest.mark.parametrize("masked", [False, True])
def test_weights_of_the_longest_table(N, masked):
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(N)
    M, d = (1 << 21) // PAGE, 64
    cache = fm.KVCache.empty(M, 1, d)
    cache.k8.copy_((torch.randn((M, 1, PAGE, d), generator=gen, device="cuda") * 96).clamp(-448, 448).to(torch.float8_e4m3fn))
    cache.kscale.fill_(2.0 ** -7)
    table = torch.randperm(M, generator=gen, device="cuda").int()[None].contiguous()
    q = torch.randn((1, 1, N, d), generator=gen, device="cuda").bfloat16()
    lens = ints([M * PAGE - 3])
    lts = None
    if masked:  # the first third and every fifth run of 1000 keys are hidden
        j = torch.arange(M * PAGE, device="cuda")
        lts = torch.where((j < M * PAGE // 3) | (j // 1000 % 5 == 2), 0, 2 ** 31 - 1).int()[None, None].contiguous()
    lse = logsums(q, cache, table, lens, 1 / 8, lts)
    old = torch.rand((M, 1, PAGE), generator=gen, device="cuda")
    for start in (None, ints([1000])):
        w = weigh(q, cache, table, lens, lse, old, start=start, lts=lts)
        s = lens - N if start is None else start
        compare(w, table, *weigh64(q, cache, table, lens, lse, old, s, 1 / 8, lts))


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,H,N", [(65535, 1, 1), (40000, 2, 17)])
def test_weights_of_the_most_sequences(B, H, N, masked):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(B)
    cache = random_cache(fm, B, 1, 64, gen)
    table = torch.randperm(B, generator=gen).int()[:, None].contiguous().cuda()
    lens = torch.randint(0, PAGE + 1, (B,), generator=gen).int().cuda()
    q = torch.randn((B, H, N, 64), generator=gen).bfloat16().cuda()
    lts = (torch.arange(PAGE) + 20).int().expand(B, 1, PAGE).contiguous().cuda() if masked else None
    lse = logsums(q, cache, table, lens, 1 / 8, lts)
    old = torch.rand((B, 1, PAGE), generator=gen).cuda()
    w = weigh(q, cache, table, lens, lse, old, lts=lts)
    for at in range(0, B, 4096):
        x = slice(at, min(B, at + 4096))
        compare(w, table[x], *weigh64(q[x], cache, table[x], lens[x], lse[x], old, (lens[x] - N).clamp(min=0), 1 / 8,
                                      None if lts is None else lts[x]))


@pytest.mark.parametrize("H,Hk,N", [(65535, 65535, 1), (60000, 15000, 9)])
def test_weights_of_the_most_heads(H, Hk, N):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(Hk)
    cache = random_cache(fm, 2, Hk, 64, gen)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    q = torch.randn((1, H, N, 64), generator=gen).bfloat16().cuda()
    lens, old = ints([100]), torch.rand((2, Hk, PAGE), generator=gen).cuda()
    lse = logsums(q, cache, table, lens, 1 / 8)
    w = weigh(q, cache, table, lens, lse, old)
    G, step = H // Hk, 3000
    for at in range(0, Hk, step):
        x, y = slice(at, min(Hk, at + step)), slice(at * G, min(Hk, at + step) * G)
        part = fm.KVCache(*(t[:, x].contiguous() for t in cache.tensors))
        compare(w[:, x], table, *weigh64(q[:, y], part, table, lens, lse[:, y], old[:, x], lens - N, 1 / 8))


def test_weights_of_more_rows_than_keys():
    fm = need_gpu()
    N, lens = 70000, ints([300])
    q, cache, table, gen = make(fm, 1, 2, 1, N, 64, [300], seed=1)
    lse = logsums(q, cache, table, lens, 1 / 8)
    old = torch.rand((cache.k8.shape[0], 1, PAGE), generator=gen).cuda()
    w = weigh(q, cache, table, lens, lse, old)
    # (the rows at positions below zero see nothing)
    table = table[:, :5].contiguous()
    want, tol = weigh64(q[:, :, N - 300:], cache, table, lens, lse[:, :, N - 300:], old, ints([0]), 1 / 8)
    compare(w, table, want, tol)


@pytest.mark.parametrize("N", [3, 50])
def test_counts_out_of_range_are_clamped(N):
    fm = need_gpu()
    lens = [200, 200, 200, 200]
    q, cache, table, gen = make(fm, 4, 4, 2, N, 64, lens, seed=N)
    wild, tame = [N + 7, -1, 2 ** 31 - 1, -2 ** 31], [N, 0, N, 0]
    old = torch.rand((cache.k8.shape[0], 2, PAGE), generator=gen).cuda()
    ws = fm.alloc_cache_weights_workspace(4, 4, 2, N, 64, table.shape[1])
    for mask in (None, mask_of("window", 4, 4, 2, N, table.shape[1] * PAGE, gen, fm)):
        lse = forward(fm, q, cache, table, lens, tame, mask)
        want = check(fm, q, cache, table, lens, tame, mask, lse=lse)
        del want
        for start, same in ((None, None), ([-5, -2 ** 31, 2 ** 31 - 1, 201], [0, 0, 200, 200])):
            got = [fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, old.clone(), ws, mask=mask, q_lens=ints(c),
                                              start=ints(s)) for c, s in ((wild, start), (tame, same))]
            assert torch.equal(*got)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


# ---------------------------------------------------------------- eviction
def steady_cache(fm, pages, Hk, d, gen):
    """A cache whose scales never change: every token has the largest code in its K and its V."""
    cache = fm.KVCache.empty(pages, Hk, d)
    step = max(1, (1 << 27) // (Hk * PAGE * d))
    for t in (cache.k8, cache.v8):
        for p in range(0, pages, step):
            shape = (min(step, pages - p),) + t.shape[1:]
            t[p:p + step] = (torch.randn(shape, generator=gen, device="cuda") * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.k8.view(torch.uint8)[..., 0] = 0x7e
    cache.v8.view(torch.uint8)[:, :, 0] = 0x7e
    return cache


def kept_positions(w, lens, n):
    """[.., most] positions of the n largest of the first lens weights, in order; 2^30 behind them."""
    j = torch.arange(w.shape[-1], device=w.device)
    order = torch.argsort(torch.where(j < lens, w, -math.inf), dim=-1, descending=True, stable=True)
    r = torch.arange(int(n.max()), device=w.device)
    return torch.where(r < n, order[..., :r.numel()], 1 << 30).sort(-1).values


def lines(cache, w, table):
    """K, V and weights of the tables' tokens: [B, Hk, M * 64, ..]."""
    t = table.long()
    k = cache.k8.view(torch.uint8)[t].transpose(1, 2).flatten(2, 3)
    v = cache.v8.view(torch.uint8)[t].permute(0, 2, 1, 4, 3).flatten(2, 3)
    return k, v, w[t].transpose(1, 2).flatten(2)


def evict_and_compare(fm, cache, table, lens, w, keep, out_table=None):
    B, Hk = table.shape[0], cache.k8.shape[1]
    ws = fm.alloc_cache_evict_workspace(B, Hk, table.shape[1])
    before = lines(cache, w, table)
    n = torch.minimum(lens, keep)
    at = kept_positions(before[2], lens[:, None, None], n[:, None, None])
    index = torch.full(at.shape, 1 << 30, dtype=torch.int32, device="cuda")
    new = fm.flashmask_cache_evict(cache, table, lens, w, keep, ws, out_table=out_table, index=index)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0) and torch.equal(new, n)
    assert torch.equal(index.long(), at)
    after = lines(cache, w, (table if out_table is None else out_table).clamp(min=0))
    there = at < 1 << 30
    at = torch.where(there, at, 0)
    for x, y in zip(before, after):
        y = y[:, :, :at.shape[2]]
        if x.dim() == 4:
            x = torch.gather(x, 2, at[..., None].expand(*at.shape, x.shape[3]))
            assert ((x == y) | ~there[..., None]).all()
        else:
            assert ((torch.gather(x, 2, at) == y) | ~there).all()
    assert (cache.kscale[table.long()] == 1).all() and (cache.vscale[table.long()] == 1).all()


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("keep", [(1 << 21) - 1, 300000])
def test_eviction_from_the_longest_table(keep, apart):
    # all but one token (in place nearly every page is written again), and an eighth
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(keep)
    M, out = (1 << 21) // PAGE, -(-keep // PAGE)
    cache = steady_cache(fm, M + (out if apart else 0), 1, 64, gen)
    w = torch.rand((cache.k8.shape[0], 1, PAGE), generator=gen, device="cuda")
    order = torch.randperm(cache.k8.shape[0], generator=gen, device="cuda").int()
    table = order[None, :M].contiguous()
    evict_and_compare(fm, cache, table, ints([M * PAGE]), w, ints([keep]), order[None, M:].contiguous() if apart else None)


@pytest.mark.parametrize("apart", [False, True])
def test_eviction_of_the_most_sequences(apart):
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(3)
    B = 65535
    cache = steady_cache(fm, 2 * B, 1, 64, gen)
    w = torch.randint(0, 50, (2 * B, 1, PAGE), generator=gen, device="cuda").float()
    order = torch.randperm(2 * B, generator=gen, device="cuda").int()[:, None].contiguous()
    lens, keep = (torch.randint(0, PAGE + 1, (B,), generator=gen, device="cuda").int() for _ in range(2))
    evict_and_compare(fm, cache, order[:B], lens, w, keep, order[B:] if apart else None)


@pytest.mark.parametrize("apart", [False, True])
def test_eviction_of_the_most_heads(apart):
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(4)
    Hk = 65535
    cache = steady_cache(fm, 3, Hk, 64, gen)
    w = torch.rand((3, Hk, PAGE), generator=gen, device="cuda")
    evict_and_compare(fm, cache, ints([[2, 0]]), ints([100]), w, ints([30]), ints([[1]]) if apart else None)


# ---------------------------------------------------------------- norm
def test_norms_past_32_bits():
    # offsets of the last head beyond 2^31 elements: each part is what it is by itself. dw: a
    # chain of 3 heads x 900 tiles, of warps, CTAs and rows, below 2^12 steps of 2^-24, and 2^-18 a term
    fm = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(5)
    H, N, d = 3, (1 << 23) + 5, 128
    x, g = (torch.empty((1, H, N, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, g):
        for h in range(H):
            for n in range(0, N, 1 << 21):
                part = t[0, h, n:n + (1 << 21)]
                part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    w = torch.rand(d, generator=gen, device="cuda") + 0.5
    freqs, _ = fm.rope_frequencies(d)
    ws = fm.alloc_norm_workspace(d)
    y, _ = fm.flashmask_norm_rope(x, None, w, None, freqs)
    dx, _, dw, _ = fm.flashmask_norm_rope_bwd(g, None, x, None, w, None, freqs, ws)
    for h in (0, H - 1):
        for n in (0, N // 2, N - 333):
            at = lambda t: t[:, h:h + 1, n:n + 333]
            pos = torch.arange(n, n + 333, dtype=torch.int32, device="cuda")[None]
            a, _ = fm.flashmask_norm_rope(at(x), None, w, None, freqs, positions=pos)
            b = fm.flashmask_norm_rope_bwd(at(g), None, at(x), None, w, None, freqs, ws, positions=pos)
            assert torch.equal(a, at(y)) and torch.equal(b[0], at(dx))
    del y, dx
    want, size = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(H):
        for n in range(0, N, 1 << 19):
            z = x[0, h, n:n + (1 << 19)].double()
            a = torch.arange(n, n + z.shape[0], device="cuda").double()[:, None] * freqs
            c, s = torch.cos(a), torch.sin(a)
            g0, g1 = g[0, h, n:n + (1 << 19)].double().split(d // 2, -1)
            u = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6)
            want += (torch.cat((g0 * c + g1 * s, g1 * c - g0 * s), -1) * u).sum(0)
            mag = g0.abs() + g1.abs()
            size += (torch.cat((mag, mag), -1) * u.abs()).sum(0)
    assert ((dw.double() - want).abs() <= size * (2.0 ** -12 + 2.0 ** -18)).all()


def test_norms_of_the_most_heads():
    fm = need_gpu()
    gen = torch.Generator().manual_seed(6)
    Hq, Hk, N, d = 40000, 25535, 2, 8
    rn = lambda h: torch.randn((1, h, N, d), generator=gen).cuda()
    q, k, dq, dk = rn(Hq), rn(Hk), rn(Hq), rn(Hk)
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=gen)).cuda() for _ in range(2))
    freqs, _ = fm.rope_frequencies(d)
    pos = torch.tensor([[7, 100000]], dtype=torch.int32, device="cuda")
    yq, yk = fm.flashmask_norm_rope(q, k, qw, kw, freqs, positions=pos)
    got = fm.flashmask_norm_rope_bwd(dq, dk, q, k, qw, kw, freqs, fm.alloc_norm_workspace(d), positions=pos)
    for y, dx, dw, x, g, w in ((yq, got[0], got[2], q, dq, qw), (yk, got[1], got[3], k, dk, kw)):
        check_forward(y, x, w, pos, freqs, False, 1.0, 1e-6)
        check_backward(dx, dw, g, x, w, pos, freqs, False, 1.0, 1e-6)
    assert f64(got[2]).shape == (d,)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from mask_aware_exact_gb300 import flashmask as fm
H, N, pages, masked = 8, {N}, {pages}, {masked}
cache = fm.KVCache.empty(pages, 2, 64)
table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
q, k = torch.randn((1, H, N, 64), device="cuda").bfloat16(), torch.randn((1, 2, N, 64), device="cuda").bfloat16()
ones = torch.ones(64, device="cuda")
held = torch.tensor([64 * pages - 100], dtype=torch.int32, device="cuda")
ws, wws = fm.alloc_cache_workspace(1, H, 2, N, 64, pages), fm.alloc_cache_weights_workspace(1, H, 2, N, 64, pages)
ews, nws = fm.alloc_cache_evict_workspace(1, 2, pages), fm.alloc_norm_workspace(64)
freqs, _ = fm.rope_frequencies(64)
lts = torch.arange(pages * 64, dtype=torch.int32, device="cuda")[None, None] + 50
mask = fm.DeviceMask(lts.contiguous(), torch.full_like(lts, 1 << 30), None, None, True) if masked else None
weights = torch.zeros((pages, 2, 64), device="cuda")
spare = [t.clone() for t in (*cache.tensors, weights)]

def step():
    q2, k2 = fm.flashmask_norm_rope(q, k, ones, ones, freqs)
    fm.flashmask_cache_append(cache, table, k2, k, held, ws)
    o, lse = fm.flashmask_fwd_cache(q2, cache, table, held + N, ws, mask=mask)
    fm.flashmask_cache_weights(q2, cache, table, held + N, lse, weights, wws, mask=mask)
    new = fm.flashmask_cache_evict(cache, table, held + N, weights, 64 * pages - 130, ews, sink=3)
    back = fm.flashmask_norm_rope_bwd(q2, k2, q, k, ones, ones, freqs, nws)
    return (o, lse, new, *back)

def state():
    return [t.clone().view(torch.uint8) for t in (*cache.tensors, weights)]

def reset():
    for t, x in zip((*cache.tensors, weights), spare):
        t.copy_(x)

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
reset()
g.replay()
torch.cuda.synchronize()
got, at = [t.clone() for t in out], state()
reset()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
assert all(torch.equal(a, b) for a, b in zip(at, state()))
for w in (ws, wws, ews):
    assert fm.flashmask_check_status(w) == (fm.FM_OK, 0)
"""


@pytest.mark.parametrize("N,pages,masked", [(1, 9, False), (4, 300, True), (40, 9, False), (40, 300, True), (1, 6000, True)])
def test_the_first_call_of_a_process_is_captured(N, pages, masked):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, N=N, pages=pages, masked=masked)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
