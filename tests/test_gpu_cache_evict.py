"""Eviction from the paged cache against the plain definition: positions, lengths,
weights, scales and codes are compared for equality (power-of-two scales make every
step exact). The refusals need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm
from oracle import evict as E

from cache_common import PAGE, cache_arrays, random_cache, random_table, values
from gpu_common import need_gpu

FAKE = 1 << 20
ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def make(fm, lens, Hk, d, seed=0, slack=1, out=None, weights="random"):
    """A cache, its table, a table of other pages for `out` tokens each, and weights."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // PAGE) for n in lens]
    out_need = [0] * len(lens) if out is None else [-(-n // PAGE) for n in out]
    pages = sum(need) + sum(out_need) + 2
    both = random_table([PAGE * (a + z) for a, z in zip(need, out_need)], max(a + z for a, z in zip(need, out_need)) + 1,
                        gen, pages=pages, device="cpu")
    table = torch.full((len(lens), max(need) + slack), 1 << 30, dtype=torch.int32)
    out_table = torch.full((len(lens), max(max(out_need), 1)), -5, dtype=torch.int32)
    for b, (a, z) in enumerate(zip(need, out_need)):
        table[b, :a] = both[b, :a]
        out_table[b, :z] = both[b, a:a + z]
    cache = random_cache(fm, pages, Hk, d, gen)
    w = torch.rand((pages, Hk, PAGE), generator=gen)
    if weights == "ties":
        w = torch.randint(0, 3, w.shape, generator=gen).float()
    elif weights == "equal":
        w = torch.ones_like(w)
    elif weights == "odd":
        odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, -1.0, 1e-42, -1e-42, 3e38, 1.0])
        w = odd[torch.randint(0, 10, w.shape, generator=gen)]
    elif weights == "tails":
        w = torch.exp(8 * torch.randn(w.shape, generator=gen))
    return cache, table.cuda(), (None if out is None else out_table.cuda()), w.cuda(), gen


def check(fm, lens, keep, Hk=2, d=64, sink=0, recent=0, apart=False, weights="random", ws=None, width=None, slack=1,
          seed=0, edit=None):
    kept = [min(n, max(k, 0)) for n, k in zip(lens, keep)]
    cache, table, out_table, w, gen = make(fm, lens, Hk, d, seed, slack, kept if apart else None, weights)
    if edit is not None:
        edit(cache, table, gen)
    B = len(lens)
    width = max(max(kept), 1) + 3 if width is None else width
    index = torch.full((B, Hk, width), -7, dtype=torch.int32, device="cuda")
    ws = fm.alloc_cache_evict_workspace(B, Hk, table.shape[1]) if ws is None else ws
    before = cache_arrays(cache) + (w.double().cpu().numpy(),)
    ln = ints(lens)
    new = fm.flashmask_cache_evict(cache, table, ln, w, ints(keep), ws, sink=sink, recent=recent,
                                   out_table=out_table, index=index)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    assert new.tolist() == kept and ln.tolist() == list(lens)
    want = E.evict(*before[:4], before[4], table.cpu().numpy(), lens, keep, sink, recent,
                   None if out_table is None else out_table.cpu().numpy())
    for b in range(B):
        for h in range(Hk):
            got = index[b, h].tolist()
            m = min(kept[b], width)
            assert got[:m] == want[5][b][h][:m] and all(x == -7 for x in got[m:]), (b, h)
    got = cache_arrays(cache) + (w.double().cpu().numpy(),)
    for x, y, name in zip(got, want[:5], ("k8", "kscale", "v8", "vscale", "weights")):
        np.testing.assert_array_equal(x, y, err_msg=name)
    return cache, table, w, new


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sink,recent", [(0, 0), (4, 10), (70, 130), (1000, 0), (0, 1000)])
def test_sizes(d, sink, recent, apart):
    fm = need_gpu()
    lens = [0, 1, 1, 63, 64, 65, 128, 200, 777, 777, 300]
    keep = [5, 1, 0, 10, 64, 64, 1, 150, 300, 776, 10000]
    check(fm, lens, keep, 2, d, sink, recent, apart)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("weights", ["ties", "equal", "odd", "tails"])
@pytest.mark.parametrize("Hk", [1, 3])
def test_weights(Hk, weights, apart):
    fm = need_gpu()
    check(fm, [500, 64, 130, 1100], [333, 1, 129, 100], Hk, 64, 3, 20, apart, weights)
    check(fm, [500, 64, 130, 1100], [333, 1, 129, 100], Hk, 64, 0, 0, apart, weights)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("slack", [1, 300, 600, 2600])
def test_clusters(slack, apart):
    # tables of more than 256, 512 and 2048 pages: clusters of 2, 4 and 8, and keys read again
    fm = need_gpu()
    check(fm, [3000, 70, 0, 1], [1111, 3, 3, 3], 1, 64, 5, 50, apart, "ties", slack=slack)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("slack", [4000, 6000])
def test_tables_far_wider_than_their_sequences(slack, apart):
    fm = need_gpu()
    check(fm, [5000, 0, 64, 1], [1200, 3, 63, 0], Hk=2, slack=slack, sink=5, recent=70, apart=apart, weights="ties")
    check(fm, [20000], [15000], Hk=1, slack=slack, sink=5, recent=700, apart=apart)


@pytest.mark.gpu
@pytest.mark.parametrize("n,keep", [(40000, 9000), (150000, 140000)])
def test_long(n, keep):
    fm = need_gpu()
    check(fm, [n, 129], [keep, 128], 1, 64, 4, 100, False, "tails", slack=0)
    check(fm, [n, 129], [n // 50, 128], 1, 64, 4, 100, True, "ties", slack=0)


@pytest.mark.gpu
def test_many_sequences():
    # more sequences than threads of a CTA
    fm = need_gpu()
    lens = [(37 * b) % 150 for b in range(700)]
    keep = [(11 * b) % 100 for b in range(700)]
    for apart in (False, True):
        check(fm, lens, keep, 1, 64, 2, 5, apart, "ties")


@pytest.mark.gpu
def test_one_token_less_each_time():
    # a cache held at its size: every call evicts one token and appends another
    fm = need_gpu()
    Hk, d, size = 2, 64, 130
    cache, table, _, w, gen = make(fm, [size + 1], Hk, d)
    ws, cw = fm.alloc_cache_evict_workspace(1, Hk, table.shape[1]), \
        fm.alloc_cache_workspace(1, Hk, Hk, 1, d, table.shape[1])
    lens = ints([size + 1])
    for step in range(20):
        before = cache_arrays(cache)
        want = E.evict(*before, w.double().cpu().numpy(), table.cpu().numpy(), [size + 1], [size], 1, 4)
        out = fm.flashmask_cache_evict(cache, table, lens, w, size, ws, sink=1, recent=4, new_lens=lens)
        assert out is lens and lens.tolist() == [size]
        for x, y in zip(cache_arrays(cache) + (w.double().cpu().numpy(),), want[:5]):
            np.testing.assert_array_equal(x, y)
        new = torch.randn((2, 1, Hk, 1, d), generator=gen).bfloat16().cuda()
        fm.flashmask_cache_append(cache, table, new[0], new[1], lens, cw)
        w[int(table[0, size // PAGE]), :, size % PAGE] = torch.rand(Hk, generator=gen).cuda()
        lens += 1
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
def test_scales_and_codes_that_are_odd(apart):
    fm = need_gpu()

    def edit(cache, table, gen):
        at = table[0, :12].tolist()
        cache.kscale[at[0]] = 2.0 ** 60
        cache.kscale[at[1]] = 2.0 ** -90   # below what e4m3 holds beside the page before
        cache.vscale[at[2]] = 0.0
        cache.kscale[at[3]] = float("nan")
        cache.vscale[at[4]] = float("inf")
        cache.kscale[at[5]] = -1.0
        cache.k8.view(torch.uint8)[at[6], :, ::9] = 0x7f  # keys that are NaN
        cache.k8.view(torch.uint8)[at[7], 0, 3, 5] = 0xff
        cache.k8[at[8]] = 0.0
        cache.v8[at[8]] = 0.0
        cache.kscale[at[9]] = 2.0 ** -126
        cache.vscale[at[9]] = 2.0 ** 127
        cache.k8[at[10]] = 2.0 ** -9  # subnormal codes
        cache.vscale[at[11]] = 2.0 ** -60
    check(fm, [760, 100], [380, 90], 2, 64, 2, 10, apart, edit=edit)
    check(fm, [760, 100], [750, 90], 2, 128, 2, 10, apart, edit=edit)


@pytest.mark.gpu
def test_budget_for_all_and_a_larger_workspace():
    fm = need_gpu()
    cache, table, _, w, _ = make(fm, [300, 20], 2, 64)
    c2 = fm.KVCache(*[t.clone() for t in cache.tensors])
    w2 = w.clone()
    ws = fm.alloc_cache_evict_workspace(5, 4, 400)
    a = fm.flashmask_cache_evict(cache, table, ints([300, 20]), w, 100, ws, sink=3)
    b = fm.flashmask_cache_evict(c2, table, ints([300, 20]), w2, ints([100, 100]), ws, sink=3)
    assert a.tolist() == b.tolist() == [100, 20] and torch.equal(w, w2)
    for x, y in zip(cache.tensors, c2.tensors):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    check(fm, [700, 65], [65, 64], 2, 128, 1, 1, True, ws=ws)
    check(fm, [700, 65], [650, 64], 4, 128, 1, 1, False, ws=ws, width=40)
    # the old table given as the new one: in place
    c3 = fm.KVCache(*[t.clone() for t in c2.tensors])
    w3 = w2.clone()
    fm.flashmask_cache_evict(c2, table, a, w2, 50, ws)
    fm.flashmask_cache_evict(c3, table, a, w3, 50, ws, out_table=table)
    assert torch.equal(w3, w2) and torch.equal(c2.k8.view(torch.uint8), c3.k8.view(torch.uint8))
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
def test_pages_past_four_gigabytes(apart):
    fm = need_gpu()
    far, lens, keep = 70000, [500, 333], [200, 333]  # 64 KB of K a page
    cache, table, out_table, w, _ = make(fm, lens, 8, 128, out=keep if apart else None)
    ws = fm.alloc_cache_evict_workspace(2, 8, table.shape[1])
    n = cache.k8.shape[0]
    big = fm.KVCache.empty(far + n, 8, 128)
    wide = torch.zeros((far + n, 8, PAGE), device="cuda")
    for x, y in zip((*big.tensors, wide), (*cache.tensors, w)):
        x[far:].view(torch.uint8).copy_(y.view(torch.uint8))
    move = lambda t: None if t is None else torch.where((t >= 0) & (t < n), t + far, t)
    fm.flashmask_cache_evict(cache, table, ints(lens), w, ints(keep), ws, sink=3, recent=9, out_table=out_table)
    ln = ints(lens)
    new = fm.flashmask_cache_evict(big, move(table), ln, wide, ints(keep), ws, sink=3, recent=9,
                                   out_table=move(out_table), new_lens=ln)
    assert new is ln and new.tolist() == keep and fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for x, y in zip((*big.tensors, wide), (*cache.tensors, w)):
        assert torch.equal(x[far:].view(torch.uint8), y.view(torch.uint8))
    assert not wide[:far].any()


@pytest.mark.gpu
def test_an_index_of_no_width_and_sizes_past_32_bits():
    fm = need_gpu()
    lens = [300, 64]
    a = check(fm, lens, [100, 64], width=0, sink=5, recent=7)
    cache, table, _, w, _ = make(fm, lens, 2, 64)
    ws = fm.alloc_cache_evict_workspace(2, 2, table.shape[1])
    new = fm.flashmask_cache_evict(cache, table, ints(lens), w, ints([100, 64]), ws, sink=5, recent=7)
    assert new.tolist() == [100, 64] and torch.equal(w, a[2])
    # more than all of it, whatever the number
    for keep, kw in ((2 ** 32 + 5, {}), (50, dict(sink=2 ** 32 + 1)), (50, dict(recent=2 ** 40))):
        cache, table, _, w, _ = make(fm, lens, 2, 64)
        old = w.clone()
        new = fm.flashmask_cache_evict(cache, table, ints(lens), w, keep, ws, **kw)
        assert new.tolist() == [min(n, keep) for n in lens]
        if keep > 300:
            assert torch.equal(w, old)
        else:
            first = table[0, 0].long()
            got = w[first, :, :50]
            pages = table[0, :5].long()
            line = old[pages].transpose(0, 1).flatten(1)[:, :300]
            assert torch.equal(got, line[:, :50] if "sink" in kw else line[:, -50:])


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
def test_streams_and_graphs(apart):
    fm = need_gpu()
    lens, keep = [900, 400, 77], [500, 399, 10]
    cache, table, out_table, w, _ = make(fm, lens, 4, 128, out=keep if apart else None)
    first = [t.clone() for t in (*cache.tensors, w)]
    ws = fm.alloc_cache_evict_workspace(3, 4, table.shape[1])
    ln, kp = ints(lens), ints(keep)
    call = lambda **kw: fm.flashmask_cache_evict(cache, table, ln, w, kp, ws, sink=2, recent=9, out_table=out_table, **kw)

    def reset():
        for t, x in zip((*cache.tensors, w), first):
            t.copy_(x)
    raw = lambda: [t.clone().view(torch.uint8) for t in (*cache.tensors, w)]
    call()
    want = raw()
    reset()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(raw(), want))
    reset()
    graphs = []
    for _ in range(2):  # two graphs that share the workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for g, out in graphs:
        reset()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(raw(), want)) and out.tolist() == keep


@pytest.mark.gpu
def test_what_is_out_of_range_is_recorded():
    fm = need_gpu()
    lens, keep = [300, 200], [150, 100]
    cache, table, out_table, w, _ = make(fm, lens, 1, 64, out=keep)
    first = [t.clone() for t in (*cache.tensors, w)]
    ws = fm.alloc_cache_evict_workspace(2, 1, table.shape[1])

    def run(**kw):
        for t, x in zip((*cache.tensors, w), first):
            t.copy_(x)
        args = dict(table=table, lens=ints(lens), keep=ints(keep), out_table=out_table)
        args.update(kw)
        fm.flashmask_cache_evict(cache, args["table"], args["lens"], w, args["keep"], ws, out_table=args["out_table"])
        return fm.flashmask_check_status(ws)[0]
    assert run() == fm.FM_OK
    good = w[out_table[1].long()].clone()
    for bad in (-1, cache.k8.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        assert run(table=t) == fm.FM_ERR_PAGE
        assert torch.equal(w[out_table[1].long()], good)
        t = out_table.clone()
        t[0, 1] = bad
        assert run(out_table=t) == fm.FM_ERR_PAGE
        assert torch.equal(w[out_table[1].long()], good)
    for n in (-1, table.shape[1] * PAGE + 1):
        assert run(lens=ints([n, 200]), table=table.clamp(max=cache.k8.shape[0] - 1), keep=ints([3, 100])) == fm.FM_ERR_PAGE
        assert torch.equal(w[out_table[1].long()], good)
    assert run(keep=ints([300, 100])) == fm.FM_ERR_PAGE  # more than the new table holds
    assert torch.equal(w[out_table[1].long()], good)
    assert run(keep=ints([-5, 100])) == fm.FM_OK
    assert run() == fm.FM_OK


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def evict(lib, k8=FAKE, v8=FAKE, kscale=FAKE, vscale=FAKE, pages=4, Hk=2, d=64, table=FAKE, max_pages=4,
          out=FAKE + 4096, out_pages=2, lens=FAKE, weights=FAKE, keep=None, budget=10, sink=0, recent=0, new_lens=FAKE,
          index=None, width=0, B=1, ws=FAKE, ws_bytes=16, cache=True):
    c = fm._FmCache(k8, v8, kscale, vscale, pages, Hk, d)
    return lib.flashmask_cache_evict(ctypes.byref(c) if cache else None, table, max_pages, out, out_pages, lens, weights,
                                     keep, budget, sink, recent, new_lens, index, width, B, ws, ws_bytes, None)


@pytest.mark.parametrize("good", [dict(), dict(out=None, out_pages=0), dict(out=FAKE, out_pages=4), dict(keep=FAKE, budget=-1),
                                  dict(index=FAKE, width=0), dict(budget=0), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)],
                         ids=str)
def test_what_is_taken(lib, good):
    assert evict(lib, **good) == fm.FM_ERR_WORKSPACE


@pytest.mark.parametrize("bad", [
    *[{n: None} for n in ("k8", "v8", "kscale", "vscale", "table", "lens", "weights", "new_lens")],
    dict(cache=False), dict(pages=0), dict(k8=FAKE + 8), dict(vscale=FAKE + 2), dict(table=FAKE + 2),
    dict(out=FAKE + 2), dict(lens=FAKE + 2), dict(weights=FAKE + 1), dict(keep=FAKE + 2), dict(new_lens=FAKE + 2),
    dict(index=FAKE + 2), dict(sink=-1), dict(recent=-1), dict(budget=-1), dict(index=FAKE, width=-1),
    dict(out=FAKE, out_pages=3)], ids=str)
def test_arguments(lib, bad):
    assert evict(lib, **bad) == fm.FM_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(d=32), dict(Hk=0), dict(B=0), dict(B=-1), dict(B=1 << 16), dict(max_pages=0),
                                 dict(max_pages=(1 << 15) + 1), dict(out_pages=0), dict(out_pages=(1 << 15) + 1)], ids=str)
def test_sizes_refused(lib, bad):
    assert evict(lib, **bad) == fm.FM_ERR_UNSUPPORTED


def test_workspace(lib):
    need = fm.flashmask_cache_evict_workspace_bytes(1, 2, 4)
    assert need > 0 and fm.flashmask_cache_evict_workspace_bytes(1, 0, 4) == 0
    for bad in (dict(ws=None, ws_bytes=need), dict(ws=FAKE + 128, ws_bytes=need), dict(ws_bytes=need - 1)):
        assert evict(lib, **bad) == fm.FM_ERR_WORKSPACE
