"""The attention weight of cached keys against the fp64 definition on the same codes,
scales and LSE; tolerances in oracle.evict.weigh. The refusals need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm
from oracle import evict as E

from cache_common import PAGE, random_cache, random_table, values
from gpu_common import need_gpu
from test_gpu_cache_fwd import make, mask_of

FAKE = 1 << 20
host = lambda t: None if t is None else t.cpu().numpy()
ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def forward(fm, q, cache, table, lens, q_lens, mask, scale=None):
    B, H, N, d = q.shape
    ws = fm.alloc_cache_workspace(B, H, cache.k8.shape[1], N, d, table.shape[1])
    lse = torch.full((B, H, N), 5.0, device="cuda")
    fm.flashmask_fwd_cache(q, cache, table, ints(lens), ws, mask=mask, q_lens=ints(q_lens), lse=lse, scale=scale)
    return lse


def check(fm, q, cache, table, lens, q_lens=None, mask=None, start=None, scale=None, lse=None, ws=None):
    B, H, N, d = q.shape
    lse = forward(fm, q, cache, table, lens, q_lens, mask, scale) if lse is None else lse
    if ws is None:
        ws = fm.alloc_cache_weights_workspace(B, H, cache.k8.shape[1], N, d, table.shape[1])
    gen = torch.Generator().manual_seed(9)
    old = torch.rand((cache.k8.shape[0], cache.k8.shape[1], PAGE), generator=gen).cuda()
    w = old.clone()
    got = fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, w, ws, mask=mask, q_lens=ints(q_lens),
                                     start=ints(start), scale=scale)
    assert got is w and fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    vec = {} if mask is None else dict(causal=mask.causal, lts=host(mask.lts), lte=host(mask.lte),
                                       uts=host(mask.uts), ute=host(mask.ute))
    want, tol = E.weigh(q.double().cpu().numpy(), values(cache.k8), host(cache.kscale), host(table), lens, q_lens,
                        host(lse), host(old), start, 1 / math.sqrt(d) if scale is None else scale, **vec)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(host(w)), nan)
    err = np.abs(host(w).astype(np.float64) - want)
    assert np.all(err[~nan] <= tol[~nan]), (err[~nan] - tol[~nan]).max()
    again = fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, old.clone(), ws, mask=mask,
                                       q_lens=ints(q_lens), start=ints(start), scale=scale)
    assert torch.equal(again.view(torch.int32), w.view(torch.int32))  # the same bits
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (8, 2), (6, 2), (16, 1), (14, 2), (40, 1)])
def test_one_token(H, Hk, d):
    fm = need_gpu()
    lens = [0, 1, 2, 63, 64, 65, 129, 700, 1500]
    q, cache, table, _ = make(fm, len(lens), H, Hk, 1, d, lens)
    check(fm, q, cache, table, lens)
    check(fm, q, cache, table, lens, start=[0, 0, 1, 60, 64, 3, 129, 64, 700])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk,N", [(4, 2, 2), (8, 1, 4), (2, 2, 9), (6, 2, 33), (4, 1, 70), (2, 2, 130),
                                    (8, 2, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens(H, Hk, N, d, causal):
    fm = need_gpu()
    lens = [N, N + 1, N + 63, 500 + N, 0]
    q_lens = [N, max(1, N - 1), 1, N, 0]
    q, cache, table, _ = make(fm, 5, H, Hk, N, d, lens, seed=N)
    mask = None if causal else fm.DeviceMask(None, None, None, None, False)
    check(fm, q, cache, table, lens, q_lens, mask)
    check(fm, q, cache, table, lens, q_lens, mask, start=[0] * 5)
    # rows at positions below zero, which see nothing when causal; no live rows
    check(fm, q, cache, table, lens, None, mask)
    check(fm, q, cache, table, lens, [0, 1, 0, 0, 0], mask, start=[1, 0, 70, 3, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["window", "window_prefix", "documents", "nothing", "upper_only", "random",
                                  "random_kv", "random_head"])
@pytest.mark.parametrize("H,Hk,N,d", [(8, 2, 1, 128), (4, 4, 1, 64), (4, 2, 5, 64), (6, 1, 40, 128),
                                      (16, 2, 1, 64), (8, 1, 33, 128)])
def test_masks(kind, H, Hk, N, d):
    fm = need_gpu()
    lens = [1 + N, 64, 333, 1000, 700]
    q, cache, table, gen = make(fm, 5, H, Hk, N, d, lens, seed=1)
    q_lens = [N, max(N - 2, 1), N, N, 1]
    mask = mask_of(kind, 5, H, Hk, N, table.shape[1] * PAGE, gen, fm)
    check(fm, q, cache, table, lens, q_lens, mask)
    check(fm, q, cache, table, lens, q_lens, mask, start=[0, 5, 100, 64, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,N", [(8, 2, 1), (4, 2, 50)])
def test_weights_of_a_row_sum_to_one(H, Hk, N):
    fm = need_gpu()
    lens = [1700, N]
    q, cache, table, _ = make(fm, 2, H, Hk, N, 128, lens)
    w = check(fm, q, cache, table, lens, start=[0, 0])
    for b, n in enumerate(lens):
        pages = table[b, :-(-n // PAGE)].long()
        per_head = w[pages].double().transpose(0, 1).flatten(1)[:, :n].sum(1)
        # LSE and the weights are each right to 2^-13 here (scores of magnitude sums below 2^5)
        assert torch.all((per_head - H // Hk * N).abs() <= H // Hk * N * 2.0 ** -12)


@pytest.mark.gpu
def test_masked_and_stale_keys_have_no_influence():
    fm = need_gpu()
    H, Hk, N, d = 4, 2, 3, 64
    lens = [100, 200]
    q, cache, table, gen = make(fm, 2, H, Hk, N, d, lens)
    L = table.shape[1] * PAGE
    lts = torch.full((2, 1, L), 2 ** 31 - 1, dtype=torch.int32)
    lts[:, :, 10:80] = 0  # hidden from every row: a whole page and parts of others
    mask = fm.DeviceMask(lts.cuda(), torch.full_like(lts, 2 ** 31 - 1).cuda(), None, None, True)
    lse = forward(fm, q, cache, table, lens, None, mask)
    clean = check(fm, q, cache, table, lens, None, mask, lse=lse)
    k = cache.k8.view(torch.uint8)
    for b in range(2):
        for j in list(range(10, 80)) + list(range(lens[b], -(-lens[b] // PAGE) * PAGE)):
            k[int(table[b, j // PAGE]), :, j % PAGE] = 0x7f
    dirty = check(fm, q, cache, table, lens, None, mask, lse=lse)
    assert torch.equal(clean, dirty)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 40])
def test_what_is_not_finite(N):
    # a NaN key spoils the rows that see it, and they every key that they see; a page
    # without a scale likewise; a query that is not finite only its own head's keys
    fm = need_gpu()
    H, Hk, d = 4, 2, 64
    lens = [130 + N, 200, 90 + N]
    q, cache, table, _ = make(fm, 3, H, Hk, N, d, lens)
    cache.k8.view(torch.uint8)[int(table[0, 1]), 0, 5] = 0x7f
    cache.kscale[int(table[1, 2]), 1] = float("inf")
    q[2, 0, 0, 3] = float("inf")
    check(fm, q, cache, table, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 3, 40])
def test_magnitudes(d, N):
    # rows from 2^-100 to 2^40 beside one another, scales from 2^-60 to 2^60, zero keys
    fm = need_gpu()
    H, Hk = 4, 1
    lens = [300]
    q, cache, table, gen = make(fm, 1, H, Hk, N, d, lens)
    e = torch.tensor([-100.0, 0.0, 3.0, 40.0])[:, None, None]
    q = (torch.randn((1, H, N, d), generator=gen) * torch.exp2(e)).bfloat16().cuda()
    cache.kscale[:, 0] = torch.exp2(torch.linspace(-60, -45, cache.k8.shape[0])).cuda()
    cache.k8[int(table[0, 1])] = 0.0
    check(fm, q, cache, table, lens)
    cache.kscale.fill_(0.0)
    check(fm, q, cache, table, lens)
    # queries so large that the factor of a score passes fp32, keys that are zero there
    q.fill_(2.0 ** 100)
    cache.kscale.fill_(2.0 ** 90)
    cache.k8.fill_(0.0)
    check(fm, q, cache, table, lens)


@pytest.mark.gpu
def test_strided_queries_and_large_workspace():
    fm = need_gpu()
    B, H, Hk, N, d = 3, 8, 2, 4, 128
    lens = [77, 500, 64]
    _, cache, table, gen = make(fm, B, H, Hk, N, d, lens)
    x = torch.randn((B, N, 3 * H * d), generator=gen).bfloat16().cuda()
    q = x[..., H * d:2 * H * d].unflatten(2, (H, d)).transpose(1, 2)
    ws = fm.alloc_cache_weights_workspace(4, 16, 4, 300, d, 64)
    a = check(fm, q, cache, table, lens, ws=ws)
    b = check(fm, q.contiguous(), cache, table, lens)
    assert torch.equal(a, b)
    check(fm, torch.randn((4, 16, 300, d), generator=gen).bfloat16().cuda(), *big(fm, gen, d), ws=ws)


def big(fm, gen, d):
    lens = [300, 301, 640, 900]
    table = random_table(lens, 64, gen)
    return random_cache(fm, int(sum(-(-n // PAGE) for n in lens)), 4, d, gen), table, lens


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 30])
def test_streams_and_graphs(N):
    fm = need_gpu()
    H, Hk, d = 8, 2, 128
    lens = [700, 1300]
    q, cache, table, _ = make(fm, 2, H, Hk, N, d, lens)
    lse = forward(fm, q, cache, table, lens, None, None)
    ws = fm.alloc_cache_weights_workspace(2, H, Hk, N, d, table.shape[1])
    ln, w0 = ints(lens), torch.rand((cache.k8.shape[0], Hk, PAGE), device="cuda")
    call = lambda w, **kw: fm.flashmask_cache_weights(q, cache, table, ln, lse, w, ws, **kw)
    want = call(w0.clone())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(w0.clone(), stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    outs, graphs = [w0.clone(), w0.clone()], []
    for w in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(w)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    call(want)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.gpu
def test_bad_pages_are_left_out():
    fm = need_gpu()
    H, Hk, N, d = 4, 2, 1, 64
    lens = [200, 130]
    q, cache, table, _ = make(fm, 2, H, Hk, N, d, lens)
    ws = fm.alloc_cache_weights_workspace(2, H, Hk, N, d, table.shape[1])
    lse = forward(fm, q, cache, table, lens, None, None)
    w = torch.rand((cache.k8.shape[0], Hk, PAGE), device="cuda")
    good = fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, w.clone(), ws)
    for bad in (-1, cache.k8.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = bad
        got = fm.flashmask_cache_weights(q, cache, t, ints(lens), lse, w.clone(), ws)
        assert fm.flashmask_check_status(ws)[0] == fm.FM_ERR_PAGE
        for p in table[1, :3].tolist():
            assert torch.equal(got[p], good[p])
        assert torch.equal(got[int(table[0, 1])], w[int(table[0, 1])])
    for n in (-1, table.shape[1] * PAGE + 1):
        fm.flashmask_cache_weights(q, cache, table.clamp(max=cache.k8.shape[0] - 1), ints([n, 130]), lse, w.clone(), ws)
        assert fm.flashmask_check_status(ws)[0] == fm.FM_ERR_PAGE
    assert torch.equal(fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, w.clone(), ws), good)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [None, "window_prefix", "documents", "random", "random_kv", "random_head"])
@pytest.mark.parametrize("H,Hk,N,d", [(8, 2, 300, 64), (3, 3, 260, 128), (33, 1, 1, 128)])
def test_many_rows(kind, H, Hk, N, d):
    # few keys for all CTAs: a group of pages is shared out by its rows
    fm = need_gpu()
    lens = [N, 1500 + N, 640]
    q, cache, table, gen = make(fm, 3, H, Hk, N, d, lens, seed=4)
    q_lens = [N, N, max(N - 135, 1)]
    mask = None if kind is None else mask_of(kind, 3, H, Hk, N, table.shape[1] * PAGE, gen, fm)
    check(fm, q, cache, table, lens, q_lens, mask)
    check(fm, q, cache, table, lens, q_lens, mask, start=[0, 70, 600])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [None, "window_prefix", "random"])
def test_a_prompt_of_its_own_keys(kind):
    # 12000 rows of one cache head, all of the sequence's tokens, and the last but one
    fm = need_gpu()
    H, N, d = 8, 1500, 64
    q, cache, table, gen = make(fm, 2, H, 1, N, d, [N, N - 1], seed=6)
    mask = None if kind is None else mask_of(kind, 2, H, 1, N, table.shape[1] * PAGE, gen, fm)
    check(fm, q, cache, table, [N, N - 1], [N, N - 1], mask)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [None, "window"])
@pytest.mark.parametrize("Hk,N", [(4, 1), (4, 11), (2, 35)])
def test_many_sequences(kind, Hk, N):
    # more segments than a CTA has threads, most of them short, some without keys
    fm = need_gpu()
    B, d = 300, 64
    gen = torch.Generator().manual_seed(N)
    lens = (torch.randint(0, 130, (B,), generator=gen) * torch.randint(0, 2, (B,), generator=gen)).tolist()
    q_lens = [min(n, N) for n in lens]
    q, cache, table, gen = make(fm, B, Hk, Hk, N, d, lens, seed=N)
    mask = None if kind is None else mask_of(kind, B, Hk, Hk, N, table.shape[1] * PAGE, gen, fm)
    check(fm, q, cache, table, lens, q_lens, mask)
    check(fm, q, cache, table, [0] * B, [0] * B, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 30])
def test_masked_on_streams_and_in_graphs(N):
    # the kernel starts beside the classification and must not read its lists too early:
    # calls whose masks differ follow one another without a pause
    fm = need_gpu()
    H, Hk, d = 8, 2, 64
    lens = [5000, 9000]
    q, cache, table, gen = make(fm, 2, H, Hk, N, d, lens)
    masks = [mask_of(k, 2, H, Hk, N, table.shape[1] * PAGE, gen, fm) for k in ("window", "random", "nothing", "documents")]
    lse = [forward(fm, q, cache, table, lens, None, m) for m in masks]
    ws = fm.alloc_cache_weights_workspace(2, H, Hk, N, d, table.shape[1])
    ln, w0 = ints(lens), torch.rand((cache.k8.shape[0], Hk, PAGE), device="cuda")
    call = lambda i, w, **kw: fm.flashmask_cache_weights(q, cache, table, ln, lse[i], w, ws, mask=masks[i], **kw)
    want = []
    for i in range(4):
        want.append(call(i, w0.clone()))
        torch.cuda.synchronize()
    outs = [w0.clone() for _ in range(40)]
    for i, w in enumerate(outs):
        call(i % 4, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    more = [w0.clone() for _ in range(4)]
    s.wait_stream(torch.cuda.current_stream())
    for i, w in enumerate(more):
        call(i, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g, held = torch.cuda.CUDAGraph(), [w0.clone() for _ in range(4)]
    with torch.cuda.graph(g):
        for i, w in enumerate(held):
            call(i, w)
    g.replay()
    for i in range(4):
        assert all(torch.equal(w, want[i]) for w in (*outs[i::4], more[i], held[i]))
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.mark.gpu
def test_bad_pages_are_left_out_with_many_rows():
    fm = need_gpu()
    H, Hk, N, d = 4, 2, 40, 64
    lens = [200, 130]
    q, cache, table, _ = make(fm, 2, H, Hk, N, d, lens)
    ws = fm.alloc_cache_weights_workspace(2, H, Hk, N, d, table.shape[1])
    lse = forward(fm, q, cache, table, lens, None, None)
    w = torch.rand((cache.k8.shape[0], Hk, PAGE), device="cuda")
    good = fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, w.clone(), ws)
    for bad in (-1, cache.k8.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = bad
        got = fm.flashmask_cache_weights(q, cache, t, ints(lens), lse, w.clone(), ws)
        assert fm.flashmask_check_status(ws)[0] == fm.FM_ERR_PAGE
        for p in [*table[1, :3].tolist(), int(table[0, 0]), int(table[0, 2])]:
            assert torch.equal(got[p], good[p])
        assert torch.equal(got[int(table[0, 1])], w[int(table[0, 1])])
    for n in (-1, table.shape[1] * PAGE + 1):
        fm.flashmask_cache_weights(q, cache, table.clamp(max=cache.k8.shape[0] - 1), ints([n, 130]), lse, w.clone(), ws)
        assert fm.flashmask_check_status(ws)[0] == fm.FM_ERR_PAGE
    assert torch.equal(fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, w.clone(), ws), good)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 30])
def test_pages_past_four_gigabytes(N):
    fm = need_gpu()
    H, Hk, d, far = 8, 8, 128, 70000  # 64 KB of K a page
    lens = [150, 333]
    q, cache, table, _ = make(fm, 2, H, Hk, N, d, lens)
    lse = forward(fm, q, cache, table, lens, None, None)
    ws = fm.alloc_cache_weights_workspace(2, H, Hk, N, d, table.shape[1])
    n = cache.k8.shape[0]
    w = torch.rand((n, Hk, PAGE), device="cuda")
    big = fm.KVCache.empty(far + n, Hk, d)
    for x, y in zip(big.tensors, cache.tensors):
        x[far:].view(torch.uint8).copy_(y.view(torch.uint8))
    wide = torch.zeros((far + n, Hk, PAGE), device="cuda")
    wide[far:] = w
    fm.flashmask_cache_weights(q, cache, table, ints(lens), lse, w, ws)
    fm.flashmask_cache_weights(q, big, torch.where(table < n, table + far, table), ints(lens), lse, wide, ws)
    assert torch.equal(wide[far:], w) and not wide[:far].any()
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def weigh(lib, k8=FAKE, v8=FAKE, kscale=FAKE, vscale=FAKE, pages=4, Hk=2, d=64, q=FAKE, qs=(256, 64, 64),
          table=FAKE, max_pages=4, lens=FAKE, q_lens=None, mask=None, B=1, H=4, N=1, scale=0.1, lse=FAKE,
          weights=FAKE, start=None, ws=FAKE, ws_bytes=16, cache=True):
    c = fm._FmCache(k8, v8, kscale, vscale, pages, Hk, d)
    m = None if mask is None else ctypes.byref(fm._FmMask(*mask))
    return lib.flashmask_cache_weights(q, None if qs is None else (ctypes.c_int64 * 3)(*qs),
                                       ctypes.byref(c) if cache else None, table, max_pages, lens, q_lens, m, B, H,
                                       N, scale, lse, weights, start, ws, ws_bytes, None)


@pytest.mark.parametrize("good", [dict(), dict(mask=(FAKE, FAKE, None, None, 1, 1)), dict(start=FAKE + 4),
                                  dict(mask=(None, None, None, None, 1, 0)), dict(q_lens=FAKE + 4),
                                  dict(weights=FAKE + 4, lse=FAKE + 4), dict(qs=(0, 0, 0))], ids=str)
def test_what_is_taken(lib, good):
    assert weigh(lib, **good) == fm.FM_ERR_WORKSPACE


@pytest.mark.parametrize("bad", [
    *[{n: None} for n in ("k8", "v8", "kscale", "vscale", "q", "qs", "table", "lens", "lse", "weights")],
    dict(cache=False), dict(pages=0), dict(k8=FAKE + 8), dict(kscale=FAKE + 2), dict(q=FAKE + 8),
    dict(table=FAKE + 2), dict(lens=FAKE + 2), dict(q_lens=FAKE + 1), dict(lse=FAKE + 2), dict(weights=FAKE + 2),
    dict(start=FAKE + 2), *[dict(qs=s) for s in ((4, 64, 64), (256, 4, 64), (256, 64, 65))],
    *[dict(scale=x) for x in (0.0, -0.1, math.inf, math.nan, 3e38)],
    *[dict(mask=m) for m in ((FAKE, None, None, None, 1, 1), (FAKE, FAKE, FAKE, None, 1, 1),
                             (FAKE + 4, FAKE, None, None, 1, 1), (None, None, FAKE, FAKE + 8, 1, 1))]], ids=str)
def test_arguments(lib, bad):
    assert weigh(lib, **bad) == fm.FM_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(d=32), dict(H=3), dict(H=0), dict(Hk=0), dict(N=0), dict(B=0), dict(max_pages=0), dict(B=-1),
    dict(max_pages=(1 << 15) + 1), dict(N=(1 << 21) + 1), dict(B=1 << 16), dict(H=1 << 16, Hk=1 << 16, N=1),
    dict(B=1 << 15, N=1 << 15), dict(mask=(FAKE, FAKE, None, None, 3, 1)), dict(mask=(FAKE, FAKE, None, None, 0, 1))],
    ids=str)
def test_sizes(lib, bad):
    assert weigh(lib, **bad) == fm.FM_ERR_UNSUPPORTED


def test_workspace(lib):
    need = fm.flashmask_cache_weights_workspace_bytes(1, 4, 2, 1, 64, 4)
    assert need > 0 and fm.flashmask_cache_weights_workspace_bytes(1, 4, 2, 1, 96, 4) == 0
    for bad in (dict(ws=None, ws_bytes=need), dict(ws=FAKE + 128, ws_bytes=need), dict(ws_bytes=need - 1)):
        assert weigh(lib, **bad) == fm.FM_ERR_WORKSPACE
