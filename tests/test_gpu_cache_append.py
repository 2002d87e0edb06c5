"""Writing into the 8-bit paged cache against the fp64 definition: codes and
scales are equal, not near. The refusals need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm
from oracle import cache as C

from cache_common import PAGE, cache_arrays, random_cache, random_table, values
from gpu_common import need_gpu

FAKE = 1 << 20


def same(a, b):
    assert np.array_equal(np.isnan(a), np.isnan(b))
    assert np.array_equal(np.nan_to_num(a), np.nan_to_num(b))


def run_and_check(fm, cache, table, k, v, start, count, ws=None, **kw):
    B, Hk, N, d = k.shape
    ws = fm.alloc_cache_workspace(B, Hk, Hk, N, d, table.shape[1]) if ws is None else ws
    f = lambda t: t.double().cpu().numpy()
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    want = C.append(*cache_arrays(cache), table.cpu().numpy(), f(k), f(v), start, count)
    fm.flashmask_cache_append(cache, table, k, v, dev(start), ws, count=dev(count), **kw)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for got, ref in zip(cache_arrays(cache), want):
        same(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk,N,start,count", [
    (1, 1, [0], None), (3, 1, [0, 1, 63, 64, 65, 127], None), (2, 2, [63, 62, 0], None),
    (2, 64, [0, 1, 64], None), (1, 65, [0, 63, 100], [65, 2, 1]), (2, 200, [17, 0, 500], [200, 0, 131]),
    (5, 7, [60, 5], [7, 3])])
@pytest.mark.parametrize("big", [1.0, 1000.0])
def test_codes_and_scales(d, Hk, N, start, count, big):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(3)
    B = len(start)
    n = [N] * B if count is None else count
    ends = [s + c for s, c in zip(start, n)]
    table = random_table(ends, 1 + max(ends) // PAGE, gen, pages=40)
    cache = random_cache(fm, 40, Hk, d, gen)
    k = (torch.randn((B, Hk, N, d), generator=gen) * big).bfloat16().cuda()
    v = (torch.randn((B, Hk, N, d), generator=gen) * big).bfloat16().cuda()
    run_and_check(fm, cache, table, k, v, start, count)
    # a second time on the same state changes nothing
    before = cache_arrays(cache)
    run_and_check(fm, cache, table, k, v, start, count)
    for a, b in zip(before, cache_arrays(cache)):
        same(a, b)


@pytest.mark.gpu
def test_token_by_token_growth():
    # one token after another, magnitudes rising and falling over many binades,
    # zeros and the smallest and largest bf16 among them
    fm = need_gpu()
    gen = torch.Generator().manual_seed(5)
    cache = random_cache(fm, 4, 2, 64, gen)
    table = torch.tensor([[3, 1]], dtype=torch.int32, device="cuda")
    scale = [0.0, 1e-38, 3e-30, 1e-5, 1.0, 448.0, 449.0, 3.3e38, 1.0, 1e-20] + [2.0 ** (i % 9) for i in range(70)]
    for t, s in enumerate(scale):
        k = (torch.randn((1, 2, 1, 64), generator=gen).clamp(-1, 1) * s).bfloat16().cuda()
        v = (torch.randn((1, 2, 1, 64), generator=gen).clamp(-1, 1) * s).bfloat16().cuda()
        run_and_check(fm, cache, table, k, v, [t], None)


@pytest.mark.gpu
def test_scale_borders():
    # absmax exactly 448 * 2^k keeps 2^k, the next bf16 above takes 2^(k + 1)
    fm = need_gpu()
    cache = fm.KVCache.empty(4, 1, 64)
    k = torch.zeros((4, 1, 1, 64))
    k[0, 0, 0, 5], k[1, 0, 0, 5], k[2, 0, 0, 5] = 448.0, 450.0, -448.0 * 2 ** 20
    table = torch.arange(4, dtype=torch.int32).view(4, 1).cuda()
    run_and_check(fm, cache, table, k.bfloat16().cuda(), (-k).bfloat16().cuda(), [0] * 4, None)
    assert torch.equal(cache.kscale[:, 0].cpu(), torch.tensor([1.0, 2.0, 2.0 ** 20, 2.0 ** -100]))
    assert cache.k8.view(torch.uint8)[0, 0, 0, 5] == 0x7e  # the largest code


@pytest.mark.gpu
def test_values_that_are_not_finite():
    fm = need_gpu()
    gen = torch.Generator().manual_seed(9)
    cache = random_cache(fm, 8, 2, 128, gen)
    table = random_table([150, 150], 4, gen, pages=8)
    k = torch.randn((2, 2, 80, 128), generator=gen).bfloat16()
    v = torch.randn((2, 2, 80, 128), generator=gen).bfloat16()
    k[0, 0, 3, 17], v[0, 1, 70, 0], k[1, 1, 0, 127], v[1, 1, 79, 64] = np.nan, np.inf, -np.inf, np.nan
    run_and_check(fm, cache, table, k.cuda(), v.cuda(), [70, 60], None)
    page = int(table[0, 1])
    got = values(cache.k8)[page, 0, 9]  # token 3 of sequence 0 sits at 73 = slot 9
    assert np.isnan(got).all() and (values(cache.v8)[page, 0, :, 9] == 0).all()
    assert np.isfinite(values(cache.v8)).all()
    # a grown scale keeps the NaN codes
    big = torch.full((2, 2, 1, 128), 1e30).bfloat16().cuda()
    run_and_check(fm, cache, table, big, big, [110, 125], None)


@pytest.mark.gpu
def test_strided_rows_stream_and_graph():
    fm = need_gpu()
    gen = torch.Generator().manual_seed(2)
    B, Hk, N, d = 3, 4, 5, 128
    qkv = torch.randn((B, N, 6 * Hk * d), generator=gen).bfloat16().cuda()
    k, v = (qkv[..., (4 + i) * Hk * d:(5 + i) * Hk * d].unflatten(2, (Hk, d)).transpose(1, 2) for i in (0, 1))
    cache = random_cache(fm, 9, Hk, d, gen)
    table = random_table([133, 70, 128], 3, gen, pages=9)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    run_and_check(fm, cache, table, k, v, [128, 62, 64], [5, 5, 4], stream=s)
    ws = fm.alloc_cache_workspace(B, Hk, Hk, N, d, 3)
    start = torch.tensor([128, 62, 64], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.flashmask_cache_append(cache, table, k, v, start, ws)
    qkv.copy_(torch.randn(qkv.shape, generator=gen))
    start.copy_(torch.tensor([0, 10, 61]))
    want = C.append(*cache_arrays(cache), table.cpu().numpy(), k.double().cpu().numpy(),
                    v.double().cpu().numpy(), [0, 10, 61], None)
    g.replay()
    for got, ref in zip(cache_arrays(cache), want):
        same(got, ref)


@pytest.mark.gpu
def test_out_of_range_is_recorded_and_left_alone():
    fm = need_gpu()
    gen = torch.Generator().manual_seed(4)
    cache = random_cache(fm, 4, 2, 64, gen)
    k = torch.randn((4, 2, 3, 64), generator=gen).bfloat16().cuda()
    ws = fm.alloc_cache_workspace(4, 2, 2, 3, 64, 2)
    before = cache_arrays(cache)
    # a page behind the last, a negative page, a negative start, no room
    table = torch.tensor([[4, 0], [-1, 0], [1, 2], [1, 2]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 5, -1, 126], dtype=torch.int32, device="cuda")
    fm.flashmask_cache_append(cache, table, k, k, start, ws)
    st, site = fm.flashmask_check_status(ws)
    assert st == fm.FM_ERR_PAGE and site in (401, 402)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for a, b in zip(before, cache_arrays(cache)):
        same(a, b)


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def call(lib, k8=FAKE, pages=4, Hk=2, d=64, k=FAKE, ks=(0, 0, 64), start=FAKE, table=FAKE, B=1, N=1,
         max_pages=4, ws=FAKE, ws_bytes=4096):
    c = fm._FmCache(k8, FAKE, FAKE, FAKE, pages, Hk, d)
    st = (ctypes.c_int64 * 3)(*ks)
    return lib.flashmask_cache_append(ctypes.byref(c), table, max_pages, k, st, FAKE, st, start, None,
                                      B, N, ws, ws_bytes, None)


def test_refusals(lib):
    for bad in (dict(k8=None), dict(k8=FAKE + 8), dict(pages=0), dict(k=None), dict(k=FAKE + 2),
                dict(ks=(0, 0, 65)), dict(start=None), dict(table=None)):
        assert call(lib, **bad) == fm.FM_ERR_INVALID_ARG, bad
    for bad in (dict(d=96), dict(B=0), dict(N=0), dict(Hk=0), dict(max_pages=0),
                dict(max_pages=(1 << 15) + 1), dict(Hk=1 << 17), dict(B=1 << 20, N=1 << 20)):
        assert call(lib, **bad) == fm.FM_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=8)):
        assert call(lib, **bad) == fm.FM_ERR_WORKSPACE, bad
    assert lib.flashmask_cache_append(None, FAKE, 4, FAKE, None, FAKE, None, FAKE, None, 1, 1, FAKE,
                                      4096, None) == fm.FM_ERR_INVALID_ARG


def test_binding_refusals():
    c = fm.KVCache.empty(2, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        c.c_struct()  # not on a GPU
    assert fm.flashmask_status_string(fm.FM_ERR_PAGE).startswith("a page")
