"""Refusals of the cached attention one by one: the call they are taken from is refused
for nothing but its workspace's size, which is looked at behind the arguments, so each
check has a case that only it can fail. Needs no GPU and launches nothing."""
import ctypes
import math

import pytest

from mask_aware_exact_gb300 import flashmask as fm

FAKE = 1 << 20
INVALID, UNSUPPORTED = fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def attend(lib, k8=FAKE, v8=FAKE, kscale=FAKE, vscale=FAKE, pages=4, Hk=2, d=64, q=FAKE, qs=(256, 64, 64),
           table=FAKE, max_pages=4, lens=FAKE, q_lens=None, mask=None, B=1, H=4, N=1, scale=0.1, o=FAKE,
           os=(256, 64, 64), lse=FAKE, ws=FAKE, ws_bytes=16, cache=True):
    c = fm._FmCache(k8, v8, kscale, vscale, pages, Hk, d)
    triple = lambda s: None if s is None else (ctypes.c_int64 * 3)(*s)
    m = None if mask is None else ctypes.byref(fm._FmMask(*mask))
    return lib.flashmask_fwd_cache(q, triple(qs), ctypes.byref(c) if cache else None, table, max_pages, lens, q_lens,
                                   m, B, H, N, scale, o, triple(os), lse, ws, ws_bytes, None)


GOOD = [dict(), dict(mask=(FAKE, FAKE, None, None, 1, 1)), dict(mask=(None, None, FAKE, FAKE, 4, 0)),
        dict(mask=(None, None, None, None, 1, 0)), dict(q_lens=FAKE + 4), dict(d=128, qs=(512, 128, 128)),
        dict(kscale=FAKE + 4, vscale=FAKE + 4), dict(qs=(0, 0, 0)), dict(scale=2.3e38)]


@pytest.mark.parametrize("good", GOOD, ids=str)
def test_what_is_taken(lib, good):
    assert attend(lib, **good) == fm.FM_ERR_WORKSPACE


@pytest.mark.parametrize("bad", [
    *[{name: None} for name in ("k8", "v8", "kscale", "vscale", "q", "qs", "table", "lens", "o", "os", "lse")],
    dict(cache=False), dict(pages=0), dict(pages=-1),
    dict(k8=FAKE + 8), dict(v8=FAKE + 8), dict(kscale=FAKE + 2), dict(vscale=FAKE + 2), dict(q=FAKE + 8),
    dict(o=FAKE + 2), dict(table=FAKE + 2), dict(lens=FAKE + 2), dict(q_lens=FAKE + 1), dict(lse=FAKE + 2),
    *[dict(qs=s) for s in ((4, 64, 64), (256, 4, 64), (256, 64, 65))],
    *[dict(os=s) for s in ((4, 64, 64), (256, 4, 64), (256, 64, 65))],
    *[dict(scale=x) for x in (0.0, -0.1, math.inf, math.nan, 3e38)],
    *[dict(mask=m) for m in ((FAKE, None, None, None, 1, 1), (None, FAKE, None, None, 1, 1),
                             (FAKE, FAKE, FAKE, None, 1, 1), (FAKE, FAKE, None, FAKE, 1, 1),
                             (FAKE + 4, FAKE, None, None, 1, 1), (FAKE, FAKE + 8, None, None, 1, 1),
                             (None, None, FAKE + 4, FAKE, 1, 1), (None, None, FAKE, FAKE + 8, 1, 1))]], ids=str)
def test_arguments(lib, bad):
    assert attend(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(d=32), dict(d=0), dict(H=3), dict(H=0), dict(Hk=0), dict(N=0), dict(B=0), dict(max_pages=0), dict(B=-1),
    dict(max_pages=(1 << 15) + 1), dict(N=(1 << 21) + 1), dict(B=1 << 16), dict(H=1 << 16, Hk=1 << 16, N=1),
    dict(B=1 << 15, N=1 << 15), dict(mask=(FAKE, FAKE, None, None, 3, 1)), dict(mask=(FAKE, FAKE, None, None, 0, 1)),
    dict(mask=(FAKE, FAKE, None, None, -1, 1))], ids=str)
def test_sizes(lib, bad):
    assert attend(lib, **bad) == UNSUPPORTED


def test_workspace(lib):
    need = fm.flashmask_cache_workspace_bytes(1, 4, 2, 1, 64, 4)
    for bad in (dict(ws=None, ws_bytes=need), dict(ws=FAKE + 128, ws_bytes=need), dict(ws_bytes=need - 1)):
        assert attend(lib, **bad) == fm.FM_ERR_WORKSPACE
