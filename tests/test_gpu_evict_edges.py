"""Eviction at its edges, against the same definition as in test_gpu_cache_evict (results
are compared for equality)."""
import pytest
import torch

from test_gpu_cache_evict import check, ints, make
from gpu_common import need_gpu


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [2.0 ** 27, 2.0 ** 28, 1.5 * 2.0 ** 100, 3.4e38])
@pytest.mark.parametrize("beside", [None, 2.0 ** -60, 2.0 ** -100])
def test_tokens_of_zeros_from_pages_of_large_scales(beside, scale, d, apart):
    # They do not count for the new page's scale, so that the old one may be more than 2^128
    # times the new: they stay zero, beside pages of small scales and where all is zero.
    fm = need_gpu()

    def edit(cache, table, gen):
        pages = table[0, :12].tolist()
        for i, page in enumerate(pages):
            if i % 3 == 1 or beside is None:
                cache.k8[page] = 0.0
                cache.v8[page] = 0.0
            if i % 3 == 1:
                cache.kscale[page] = scale
                cache.vscale[page] = scale
            elif beside is not None:
                cache.kscale[page] = beside
                cache.vscale[page] = beside
        cache.k8.view(torch.uint8)[pages[4], :, ::2] = 0x80  # of either sign
    check(fm, [760, 100], [380, 90], 2, d, 2, 10, apart, edit=edit)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
def test_zeros_beside_a_large_token_that_is_given_up(apart):
    # equal weights: positions 0 .. 49 stay and the last 100, so that the token of page 3 which
    # set its scale goes and zeros of that page move to another
    fm = need_gpu()

    def edit(cache, table, gen):
        cache.k8.zero_()
        cache.v8.zero_()
        page = int(table[0, 3])
        cache.k8[page, :, 0, 5] = 300.0
        cache.v8[page, :, 7, 1] = -300.0
        cache.kscale[page] = 2.0 ** 40
        cache.vscale[page] = 2.0 ** 28
    check(fm, [300], [150], 2, 64, 0, 100, apart, "equal", edit=edit)


@pytest.mark.gpu
def test_sizes_below_zero():
    # of one sequence they count as zero; for all of them they are refused, as the header says
    fm = need_gpu()
    cache, table, _, w, _ = make(fm, [100, 64], 2, 64)
    ws = fm.alloc_cache_evict_workspace(2, 2, table.shape[1])
    first = [t.clone() for t in (*cache.tensors, w)]
    for keep in (-1, -5, -2 ** 40):
        with pytest.raises(fm.FlashMaskError):
            fm.flashmask_cache_evict(cache, table, ints([100, 64]), w, keep, ws)
    for kw in (dict(sink=-1), dict(recent=-2 ** 33)):
        with pytest.raises(fm.FlashMaskError):
            fm.flashmask_cache_evict(cache, table, ints([100, 64]), w, 10, ws, **kw)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*cache.tensors, w), first))
    assert fm.flashmask_cache_evict(cache, table, ints([100, 64]), w, ints([-5, 64]), ws).tolist() == [0, 64]
    assert fm.flashmask_cache_evict(cache, table, ints([0, 64]), w, 0, ws).tolist() == [0, 0]


# Tables of more than 8 x 704 pages: the selection reads the weights again in each pass.
WIDE = 6000


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("weights", ["odd", "equal", "tails"])
def test_weights_of_any_value_in_tables_that_are_not_held(weights, apart):
    fm = need_gpu()
    check(fm, [3000, 70, 0, 1], [1111, 3, 3, 3], 2, 64, 5, 50, apart, weights, slack=WIDE)
    check(fm, [3000, 65], [17, 64], 1, 128, 0, 0, apart, weights, slack=WIDE)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_a_page_that_is_not_there_in_wide_tables(bad):
    # its keys count as NaN, so that they are the first to go, as in a table whose keys are held;
    # the other sequence is cut down as ever
    fm = need_gpu()
    lens, keep = [3000, 700], [1500, 100]
    cache, table, out_table, w, _ = make(fm, lens, 2, 64, out=keep, weights="odd")
    first = [t.clone() for t in (*cache.tensors, w)]
    got = []
    for width in (table.shape[1], WIDE):
        for missing in (False, True):
            t = torch.full((2, width), 1 << 30, dtype=torch.int32, device="cuda")
            t[:, :table.shape[1]] = table
            if missing:
                t[0, 20] = bad
            ws = fm.alloc_cache_evict_workspace(2, 2, width)
            for x, y in zip((*cache.tensors, w), first):
                x.copy_(y)
            index = torch.full((2, 2, keep[0]), -7, dtype=torch.int32, device="cuda")
            new = fm.flashmask_cache_evict(cache, t, ints(lens), w, ints(keep), ws, sink=3, recent=9,
                                           out_table=out_table, index=index)
            assert new.tolist() == keep
            # none of the missing page's tokens is kept, so that nothing of it is moved, but it
            # was looked at
            assert fm.flashmask_check_status(ws)[0] == (fm.FM_ERR_PAGE if missing else fm.FM_OK)
            gone = ((index[0] >= 20 * 64) & (index[0] < 21 * 64)).sum()
            assert (int(gone) == 0) == missing
            got.append([x.clone().view(torch.uint8) for x in (*cache.tensors, w, index)])
    for x, y in zip(got[:2], got[2:]):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    for a, b in zip(got[0][:5], got[1][:5]):  # the other sequence's pages
        at = out_table[1, :2].long()
        assert torch.equal(a[at], b[at])
