"""A cache's checked handle (sizes and pointers that the kernels take as they are)
follows its tensors when they are changed in place, at the same address too: a
stale page count or stride would let the kernels leave the tensors."""
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm

from gpu_common import need_gpu

PAGES, HK, D = 6, 2, 64


def fewer_pages(t):
    t.set_(t[:PAGES // 2])


def other_heads(t):
    t.set_(t.view((PAGES * HK, 1) + t.shape[2:]))


def smaller(t):
    t.resize_((1,) + t.shape[1:])


def other_layout(t):
    t.transpose_(-1, -2)


def other_type(t):
    t.data = t.data.view(torch.uint8 if t.element_size() == 1 else torch.int32)


CHANGES = [fewer_pages, other_heads, smaller, other_layout, other_type]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("change", CHANGES)
def test_a_change_in_place_is_checked_again(which, change, monkeypatch):
    monkeypatch.setattr(fm.KVCache, "_check", lambda c: [(t.shape, t.stride(), t.dtype) for t in c.tensors])
    c = fm.KVCache.empty(PAGES, HK, D, device="cpu")
    first = c._handle
    assert c._handle is first  # nothing changed: the handle is kept
    t = c.tensors[which]
    at = t.data_ptr()
    change(t)
    assert t.data_ptr() == at
    assert c._handle == c._check() != first


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("change", CHANGES)
def test_a_changed_tensor_is_refused(which, change):
    need_gpu()
    c = fm.KVCache.empty(PAGES, HK, D)
    ws = fm.alloc_cache_workspace(1, HK, HK, 1, D, PAGES)
    k = torch.zeros((1, HK, 1, D), device="cuda").bfloat16()
    table = torch.arange(PAGES, dtype=torch.int32, device="cuda")[None]
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    fm.flashmask_cache_append(c, table, k, k, start, ws)
    change(c.tensors[which])
    with pytest.raises(ValueError):
        fm.flashmask_cache_append(c, table, k, k, start, ws)
    with pytest.raises(ValueError):
        fm.flashmask_fwd_cache(k, c, table, start + 1, ws)


@pytest.mark.gpu
def test_a_cache_cut_to_fewer_pages():
    # all four tensors cut alike at the same address: a page behind the new end is
    # recorded, not read
    need_gpu()
    c = fm.KVCache.empty(PAGES, HK, D)
    ws = fm.alloc_cache_workspace(1, HK, HK, 1, D, PAGES)
    q = torch.ones((1, HK, 1, D), device="cuda").bfloat16()
    table = torch.arange(PAGES, dtype=torch.int32, device="cuda")[None]
    lens = torch.full((1,), 64 * PAGES, dtype=torch.int32, device="cuda")
    fm.flashmask_fwd_cache(q, c, table, lens, ws)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for t in c.tensors:
        fewer_pages(t)
    assert c.c_struct().pages == PAGES // 2
    fm.flashmask_fwd_cache(q, c, table, lens, ws)
    assert fm.flashmask_check_status(ws)[0] == fm.FM_ERR_PAGE
