"""Attention over the 8-bit paged cache against the fp64 definition on the same
codes and scales; tolerances in cache_common.attention_bounds. The refusals need
no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm
from oracle import cache as C

from cache_common import PAGE, attention_bounds, cache_arrays, random_cache, random_table
from gpu_common import need_gpu

FAKE = 1 << 20
MARK = 123.0  # what O and LSE hold before a call


def run(fm, q, cache, table, lens, q_lens=None, mask=None, scale=None, ws=None, **kw):
    B, H, N, d = q.shape
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = fm.alloc_cache_workspace(B, H, cache.k8.shape[1], N, d, table.shape[1]) if ws is None else ws
    o = torch.full((B, H, N, d), MARK, device="cuda").bfloat16()
    lse = torch.full((B, H, N), MARK, device="cuda")
    fm.flashmask_fwd_cache(q, cache, table, dev(lens), ws, mask=mask, q_lens=dev(q_lens), scale=scale,
                           o=o, lse=lse, **kw)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    return o, lse


def check(o, lse, q, cache, table, lens, q_lens=None, mask=None, scale=None, nan_rows=()):
    B, H, N, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    host = lambda t: None if t is None else t.cpu().numpy()
    vec = {} if mask is None else dict(causal=mask.causal, lts=host(mask.lts), lte=host(mask.lte),
                                       uts=host(mask.uts), ute=host(mask.ute))
    arrays = cache_arrays(cache)
    f = lambda t: t.double().cpu().numpy()
    ref = C.attend(f(q), *arrays, table.cpu().numpy(), lens, q_lens, scale, **vec)
    tol_o, tol_l = attention_bounds(ref, max(max(lens), 1))
    go, gl = f(o), f(lse)
    for b in range(B):
        live = N if q_lens is None else q_lens[b]
        assert (go[b, :, live:] == MARK).all() and (gl[b, :, live:] == MARK).all()
        for h in range(H):
            for t in range(live):
                if (b, h, t) in nan_rows:
                    assert np.isnan(go[b, h, t]).all() and np.isnan(gl[b, h, t])
                    continue
                if np.isneginf(ref[1][b, h, t]):
                    assert (go[b, h, t] == 0).all() and np.isneginf(gl[b, h, t]), (b, h, t)
                    continue
                assert abs(gl[b, h, t] - ref[1][b, h, t]) <= tol_l[b, h, t], (b, h, t)
                err = np.abs(go[b, h, t] - ref[0][b, h, t])
                assert np.all(err <= tol_o[b, h, t]), (b, h, t, (err - tol_o[b, h, t]).max())


def make(fm, B, H, Hk, N, d, lens, seed=0, slack=1, qscale=1.0):
    gen = torch.Generator().manual_seed(seed)
    most = max(1, -(-max(lens) // PAGE)) + slack
    pages = sum(-(-n // PAGE) for n in lens) + 2
    table = random_table(lens, most, gen, pages=pages)
    cache = random_cache(fm, pages, Hk, d, gen)
    q = (torch.randn((B, H, N, d), generator=gen) * qscale).bfloat16().cuda()
    return q, cache, table, gen


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (8, 2), (6, 2), (16, 1), (14, 2), (40, 1)])
def test_one_token(H, Hk, d):
    fm = need_gpu()
    lens = [0, 1, 2, 63, 64, 65, 129, 700, 1500]
    q, cache, table, _ = make(fm, len(lens), H, Hk, 1, d, lens)
    o, lse = run(fm, q, cache, table, lens)
    check(o, lse, q, cache, table, lens)


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
    o, lse = run(fm, q, cache, table, lens, q_lens, mask)
    check(o, lse, q, cache, table, lens, q_lens, mask)
    # without q_lens every row is real, the first ones of a sequence shorter
    # than N at positions below zero, which see nothing when causal
    o, lse = run(fm, q, cache, table, lens, None, mask)
    check(o, lse, q, cache, table, lens, None, mask)


def mask_of(kind, B, H, Hk, N, L, gen, fm):
    j = torch.arange(L, dtype=torch.int32)
    none = torch.zeros((B, 1, L), dtype=torch.int32)
    if kind == "window":
        lts = (j + 50).expand(B, 1, L).contiguous()
        m = (lts, torch.full_like(lts, L), None, None, True)
    elif kind == "window_prefix":
        lts = torch.where(j < 20, L, j + 70).to(torch.int32).expand(B, 1, L).contiguous()
        m = (lts, torch.full_like(lts, 2 ** 31 - 1), None, None, True)
    elif kind == "documents":
        lts = ((j // 100 + 1) * 100).to(torch.int32).expand(B, 1, L).contiguous()
        m = (lts, torch.full_like(lts, L), none, (j // 100 * 100).to(torch.int32).expand(B, 1, L).contiguous(), False)
    elif kind == "nothing":
        m = (none, torch.full_like(none, 2 ** 31 - 1), None, None, True)
    elif kind == "upper_only":
        m = (None, None, none, torch.full_like(none, L // 3), True)
    else:  # random bounds per head, empty, reversed and extreme ones among them
        Hm = {"random": 1, "random_kv": Hk, "random_head": H}[kind]
        r = lambda: torch.randint(-30, L + 30, (B, Hm, L), generator=gen).int()
        m = [r(), r(), r(), r(), True]
        m[0][..., ::7], m[1][..., ::11] = -2 ** 31, 2 ** 31 - 1
        m[2][..., ::3] = 2 ** 31 - 1
    return fm.DeviceMask(*[None if t is None else t.cuda() for t in m[:4]], m[4])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["window", "window_prefix", "documents", "nothing", "upper_only", "random",
                                  "random_kv", "random_head"])
@pytest.mark.parametrize("H,Hk,N,d", [(8, 2, 1, 128), (4, 4, 1, 64), (4, 2, 5, 64), (6, 1, 40, 128),
                                      (16, 2, 1, 64)])
def test_masks(kind, H, Hk, N, d):
    fm = need_gpu()
    lens = [1 + N, 64, 333, 1000, 700]
    q, cache, table, gen = make(fm, 5, H, Hk, N, d, lens, seed=1)
    q_lens = [N, max(N - 2, 1), N, N, 1]
    mask = mask_of(kind, 5, H, Hk, N, table.shape[1] * PAGE, gen, fm)
    o, lse = run(fm, q, cache, table, lens, q_lens, mask)
    check(o, lse, q, cache, table, lens, q_lens, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 20, 150])
def test_masked_and_stale_codes_have_no_influence(N):
    # NaN codes behind the end of a sequence and in unused pages, a poisoned
    # token: only rows that see the poisoned token become NaN
    fm = need_gpu()
    lens = [200, 70 + N]
    q, cache, table, gen = make(fm, 2, 4, 2, N, 128, lens, seed=6)
    k8, v8 = cache.k8.view(torch.uint8), cache.v8.view(torch.uint8)
    used = set()
    for b, n in enumerate(lens):
        for i in range(-(-n // PAGE)):
            p = int(table[b, i])
            used.add(p)
            live = min(PAGE, n - i * PAGE)
            k8[p, :, live:] = 0x7f
            v8[p, :, :, live:] = 0xff
    for p in range(k8.shape[0]):
        if p not in used:
            k8[p], v8[p] = 0xff, 0x7f
            cache.kscale[p] = cache.vscale[p] = float("nan")
    o, lse = run(fm, q, cache, table, lens)
    check(o, lse, q, cache, table, lens)
    # poison key 100 of sequence 0, head 1 of the cache (query heads 2 and 3)
    p = int(table[0, 1])
    k8[p, 1, 100 - PAGE], v8[p, 1, :, 100 - PAGE] = 0x7f, 0
    o, lse = run(fm, q, cache, table, lens)
    bad = {(0, h, t) for h in (2, 3) for t in range(N) if 200 - N + t >= 100}
    check(o, lse, q, cache, table, lens, nan_rows=bad)
    # masked for every row, or for some
    L = table.shape[1] * PAGE
    lts = torch.full((2, 1, L), L, dtype=torch.int32)
    lts[0, 0, 100] = 200 - N + N // 2  # hidden from the later half of the rows
    mask = fm.DeviceMask(lts.cuda(), torch.full_like(lts, L).cuda(), None, None, True)
    o, lse = run(fm, q, cache, table, lens, mask=mask)
    bad = {(0, h, t) for h in (2, 3) for t in range(N // 2) if 200 - N + t >= 100}
    check(o, lse, q, cache, table, lens, mask=mask, nan_rows=bad)


@pytest.mark.gpu
def test_query_rows_that_are_not_finite():
    fm = need_gpu()
    for N in (3, 140):
        lens = [300]
        q, cache, table, _ = make(fm, 1, 4, 2, N, 64, lens)
        q[0, 1, 0, 5], q[0, 2, 1, 63], q[0, 3, 2, 0] = float("nan"), float("inf"), -float("inf")
        o, lse = run(fm, q, cache, table, lens)
        bad = {(0, 1, 0), (0, 2, 1), (0, 3, 2)}
        q2 = q.clone()
        for b, h, t in bad:
            q2[b, h, t] = 0
        check(o, lse, q2, cache, table, lens, nan_rows=bad)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 6, 140])
def test_scales_far_apart(N):
    # one page's values are 2^60 times the others', seen or hidden; attention
    # concentrated on pages whose value scale is tiny; extreme scales
    fm = need_gpu()
    lens = [400, 400, 400]
    q, cache, table, _ = make(fm, 3, 4, 2, N, 128, lens, seed=8)
    t = table.cpu()
    cache.vscale[t[0, 3].item()] = 2.0 ** 60
    cache.vscale[t[1, 2].item()] = 2.0 ** -90
    cache.vscale[t[2, :7].long().cuda()] = 2.0 ** -100
    cache.kscale[t[2, 1].item()] = 2.0 ** -100
    L = table.shape[1] * PAGE
    lts = torch.full((3, 1, L), L, dtype=torch.int32)
    lts[0, 0, 3 * PAGE:4 * PAGE] = 0  # the page with huge values is hidden in sequence 0
    lts[1, 0, :2 * PAGE] = 0
    lts[1, 0, 3 * PAGE:] = 0          # only the tiny page is visible in sequence 1
    for mask in (None, fm.DeviceMask(lts.cuda(), torch.full_like(lts, L).cuda(), None, None, True)):
        o, lse = run(fm, q, cache, table, lens, mask=mask)
        check(o, lse, q, cache, table, lens, mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("qscale", [0.0, 1e-30, 30.0, 1e4])
def test_query_magnitudes(qscale):
    # all keys equal weight (q = 0), tiny scores, one key taking all the weight
    fm = need_gpu()
    for N in (1, 140):
        lens = [257, 1000]
        q, cache, table, _ = make(fm, 2, 8, 2, N, 128, lens, seed=2, qscale=qscale)
        o, lse = run(fm, q, cache, table, lens)
        check(o, lse, q, cache, table, lens)


@pytest.mark.gpu
def test_mixed_magnitudes_within_a_query():
    # small elements beside large ones still count: keys that are zero where the
    # query is large
    fm = need_gpu()
    lens = [200]
    for N in (1, 140):
        q, cache, table, _ = make(fm, 1, 2, 1, N, 64, lens, seed=4)
        q[..., :8] = 2048.0
        cache.k8.view(torch.uint8)[..., :8] = 0
        o, lse = run(fm, q, cache, table, lens, scale=1.0)
        check(o, lse, q, cache, table, lens, scale=1.0)


@pytest.mark.gpu
def test_strides_streams_and_repeatability():
    fm = need_gpu()
    B, H, Hk, N, d = 3, 8, 2, 6, 128
    lens = [1000, 90, 2000]
    q, cache, table, _ = make(fm, B, H, Hk, N, d, lens)
    o, lse = run(fm, q, cache, table, lens)
    check(o, lse, q, cache, table, lens)
    # token-major Q and O
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    ot = torch.zeros((B, N, H, d), device="cuda").bfloat16().transpose(1, 2)
    lt = torch.zeros((B, H, N), device="cuda")
    ws = fm.alloc_cache_workspace(B, H, Hk, N, d, table.shape[1])
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fm.flashmask_fwd_cache(qt, cache, table, ld, ws, o=ot, lse=lt)
    assert torch.equal(ot, o) and torch.equal(lt, lse)
    # the same bits again, on another stream and on a used workspace
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        o2, l2 = fm.flashmask_fwd_cache(q, cache, table, ld, ws, stream=s)
        s.synchronize()
        assert torch.equal(o2, o) and torch.equal(l2, lse)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 5, 70])
def test_output_over_the_query(N):
    fm = need_gpu()
    lens = [700 + N, 64 * 90, N]
    q, cache, table, _ = make(fm, 3, 8, 2, N, 128, lens, seed=3)
    o, lse = run(fm, q, cache, table, lens)
    ws = fm.alloc_cache_workspace(3, 8, 2, N, 128, table.shape[1])
    o2, lse2 = fm.flashmask_fwd_cache(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), ws, o=q)
    assert o2.data_ptr() == q.data_ptr() and torch.equal(o, q) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_a_cache_whose_storage_has_moved():
    """A handle made before its tensor got another storage reads the new one."""
    fm = need_gpu()
    lens = [200]
    q, cache, table, gen = make(fm, 1, 4, 2, 1, 64, lens, seed=4)
    run(fm, q, cache, table, lens)
    other = random_cache(fm, cache.k8.shape[0], 2, 64, gen)
    cache.k8.set_(other.k8)
    o, lse = run(fm, q, cache, table, lens)
    check(o, lse, q, cache, table, lens)


@pytest.mark.gpu
def test_one_workspace_serves_all_sizes_in_turn():
    fm = need_gpu()
    ws = fm.alloc_cache_workspace(8, 32, 4, 40, 128, 40)
    g = torch.Generator().manual_seed(0)
    for i, (B, H, Hk, N, d, L, masked) in enumerate([
            (1, 8, 1, 1, 128, 2400, False), (8, 32, 4, 1, 64, 700, True), (2, 8, 2, 40, 128, 2000, False),
            (1, 1, 1, 1, 64, 2500, False), (3, 16, 4, 8, 128, 900, True), (1, 8, 1, 1, 128, 2400, False),
            (1, 32, 1, 9, 64, 2000, True)]):
        lens = [max(N, L - 97 * b) for b in range(B)]
        q, cache, table, _ = make(fm, B, H, Hk, N, d, lens, seed=i)
        mask = mask_of("window_prefix", B, H, Hk, N, table.shape[1] * PAGE, g, fm) if masked else None
        o, lse = run(fm, q, cache, table, lens, mask=mask, ws=ws)
        check(o, lse, q, cache, table, lens, mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("masked", [False, True])
def test_graph_replay_with_other_lengths(masked):
    # one capture serves a growing batch: lengths and pages live on the device
    fm = need_gpu()
    B, H, Hk, N, d = 4, 8, 2, 1, 128
    full = [900, 1200, 64, 700]
    q, cache, table, _ = make(fm, B, H, Hk, N, d, full)
    ws = fm.alloc_cache_workspace(B, H, Hk, N, d, table.shape[1])
    lens = torch.tensor(full, dtype=torch.int32, device="cuda")
    L = table.shape[1] * PAGE
    lts = (torch.arange(L) + 300).int().expand(B, 1, L).contiguous().cuda()
    mask = fm.DeviceMask(lts, torch.full_like(lts, L), None, None, True) if masked else None
    fm.flashmask_fwd_cache(q, cache, table, lens, ws, mask=mask)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = fm.flashmask_fwd_cache(q, cache, table, lens, ws, mask=mask)
    for now in (full, [1, 1200, 0, 65], [0, 0, 0, 0], [899, 3, 64, 1]):
        lens.copy_(torch.tensor(now))
        g.replay()
        check(o, lse, q, cache, table, now, mask=mask)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 140])
def test_long_sequence(N):
    fm = need_gpu()
    lens = [40000]
    q, cache, table, _ = make(fm, 1, 2, 1, N, 64, lens)
    o, lse = run(fm, q, cache, table, lens, [N])
    check(o, lse, q, cache, table, lens, [N])


@pytest.mark.gpu
@pytest.mark.parametrize("H,N,d,lens", [
    (4, 1, 64, [64 * 700]), (4, 1, 128, [64 * 230 + 5, 64 * 60]), (6, 3, 64, [30000, 100, 0]),
    (2, 40, 64, [64 * 420]), (1, 140, 128, [64 * 330 + 1]), (3, 50, 128, [20000, 64 * 40, 9000])])
def test_sequences_cut_into_many_parts(H, N, d, lens):
    """Enough parts of one segment that they are added up in groups first; the counters
    are back at zero afterwards, so that a second call gives the same bits."""
    fm = need_gpu()
    q, cache, table, _ = make(fm, len(lens), H, 1, N, d, lens, seed=7)
    ws = fm.alloc_cache_workspace(len(lens), H, 1, N, d, table.shape[1])
    o, lse = run(fm, q, cache, table, lens, ws=ws)
    check(o, lse, q, cache, table, lens)
    o2, lse2 = run(fm, q, cache, table, lens, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hk,N,d,kind,most", [
    (280, 8, 4, 1, 64, None, 330), (140, 16, 8, 2, 128, "window_prefix", 330), (140, 16, 8, 1, 128, None, 330),
    (600, 4, 2, 5, 64, "documents", 330), (140, 8, 8, 1, 64, None, 64), (1100, 1, 1, 3, 128, "documents", 100)])
def test_many_short_sequences(B, H, Hk, N, d, kind, most):
    """More segments than warps, among them empty ones and a page out of range: each
    is one warp's. With a page or two for each segment the last CTAs have none."""
    fm = need_gpu()
    gen = torch.Generator().manual_seed(B)
    lens = [0 if b % 17 == 3 else 1 + int(x) for b, x in enumerate(torch.randint(0, most, (B,), generator=gen))]
    q_lens = [min(N, n) for n in lens]
    q, cache, table, gen = make(fm, B, H, Hk, N, d, lens, seed=B)
    mask = None
    if kind is not None:
        mask = mask_of(kind, B, H, Hk, N, table.shape[1] * PAGE, gen, fm)
    ws = fm.alloc_cache_workspace(B, H, Hk, N, d, table.shape[1])
    o, lse = run(fm, q, cache, table, lens, q_lens, mask, ws=ws)
    check(o, lse, q, cache, table, lens, q_lens, mask)
    o2, lse2 = run(fm, q, cache, table, lens, q_lens, mask, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # a page out of range in one sequence is recorded if one of its keys is visible (no
    # other entry is read); the others keep their results
    bad = next(b for b, n in enumerate(lens) if n > most * 3 // 5)
    at = 1 if most > 200 else 0
    table[bad, at] = cache.k8.shape[0]
    lens_d, q_d = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, q_lens))
    o3, _ = fm.flashmask_fwd_cache(q, cache, table, lens_d, ws, mask=mask, q_lens=q_d,
                                   o=torch.full_like(o, MARK))
    i = np.arange(lens[bad] - q_lens[bad], lens[bad])[:, None]
    j = np.arange(PAGE * at, PAGE * (at + 1))
    see = np.repeat(j[None] < lens[bad], len(i), 0) if mask is not None and not mask.causal else j <= i  # (i < lens)
    if mask is not None:
        vec = lambda t: t[bad, 0, PAGE * at:PAGE * (at + 1)].cpu().numpy()
        see &= ~((vec(mask.lts) <= i) & (i < vec(mask.lte)))
        if mask.uts is not None:
            see &= ~((vec(mask.uts) <= i) & (i < vec(mask.ute)))
    assert fm.flashmask_check_status(ws)[0] == (fm.FM_ERR_PAGE if see.any() else fm.FM_OK)
    keep = [b for b in range(B) if b != bad]
    assert torch.equal(o3[keep], o[keep])


@pytest.mark.gpu
def test_codes_behind_two_gigabytes():
    # pages whose offset passes 2^31 bytes
    fm = need_gpu()
    Hk, d = 16, 128
    pages = (1 << 31) // (Hk * PAGE * d) + 40
    cache = fm.KVCache.empty(pages, Hk, d)
    gen = torch.Generator().manual_seed(0)
    small = random_cache(fm, 4, Hk, d, gen)
    at = [pages - 1, 0, pages - 9, 3]
    for i, p in enumerate(at):
        cache.k8.view(torch.uint8)[p] = small.k8.view(torch.uint8)[i]
        cache.v8.view(torch.uint8)[p] = small.v8.view(torch.uint8)[i]
        cache.kscale[p], cache.vscale[p] = small.kscale[i], small.vscale[i]
    q = torch.randn((1, Hk, 1, d), generator=gen).bfloat16().cuda()
    far = torch.tensor([at], dtype=torch.int32, device="cuda")
    near = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for N in (1, 200):
        qq = q.expand(1, Hk, N, d).contiguous()
        a, la = run(fm, qq, cache, far, [250])
        b, lb = run(fm, qq, small, near, [250])
        assert torch.equal(a, b) and torch.equal(la, lb)
        check(b, lb, qq, small, near, [250])
    # and written there
    k = torch.randn((1, Hk, 1, d), generator=gen).bfloat16().cuda()
    ws = fm.alloc_cache_workspace(1, Hk, Hk, 1, d, 4)
    for c, t in ((cache, far), (small, near)):
        fm.flashmask_cache_append(c, t, k, k, torch.tensor([10], dtype=torch.int32, device="cuda"), ws)
    assert torch.equal(cache.k8.view(torch.uint8)[at[0]], small.k8.view(torch.uint8)[0])
    assert torch.equal(cache.v8.view(torch.uint8)[at[0]], small.v8.view(torch.uint8)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 140])
def test_out_of_range_is_recorded(N):
    fm = need_gpu()
    lens = [200, 200]
    q, cache, table, _ = make(fm, 2, 4, 2, N, 64, lens)
    want = run(fm, q, cache, table, lens)
    for bad in (cache.k8.shape[0], -1, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad
        ws = fm.alloc_cache_workspace(2, 4, 2, N, 64, table.shape[1])
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, lse = fm.flashmask_fwd_cache(q, cache, t, ld, ws)
        assert fm.flashmask_check_status(ws) == (fm.FM_ERR_PAGE, 404)
        assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])
        # the workspace serves on
        o, lse = fm.flashmask_fwd_cache(q, cache, table, ld, ws)
        assert torch.equal(o, want[0]) and fm.flashmask_check_status(ws) == (fm.FM_OK, 0)
    for n in (-1, table.shape[1] * PAGE + 1):
        ld = torch.tensor([n, 200], dtype=torch.int32, device="cuda")
        o, lse = fm.flashmask_fwd_cache(q, cache, table.clamp(max=cache.k8.shape[0] - 1), ld, ws)
        assert fm.flashmask_check_status(ws) == (fm.FM_ERR_PAGE, 403)
        # sequence 1 is right; its bits may differ, because the line of pages is
        # cut elsewhere when another sequence's length changes
        check(o[1:], lse[1:], q[1:], cache, table[1:], lens[1:])


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def call(lib, q=FAKE, qs=(0, 0, 64), k8=FAKE, pages=4, Hk=2, d=64, H=4, N=1, B=1, max_pages=4, lens=FAKE,
         mask=None, scale=0.1, o=FAKE, ws=FAKE, ws_bytes=1 << 30):
    c = fm._FmCache(k8, FAKE, FAKE, FAKE, pages, Hk, d)
    st = (ctypes.c_int64 * 3)(*qs)
    return lib.flashmask_fwd_cache(q, st, ctypes.byref(c), FAKE, max_pages, lens, None,
                                   None if mask is None else ctypes.byref(mask), B, H, N, scale, o, st,
                                   FAKE, ws, ws_bytes, None)


def test_refusals(lib):
    half = fm._FmMask(FAKE, None, None, None, 1, 1)
    upper = fm._FmMask(FAKE, FAKE, None, FAKE, 1, 1)
    for bad in (dict(q=None), dict(q=FAKE + 8), dict(qs=(0, 4, 64)), dict(k8=None), dict(pages=0),
                dict(lens=None), dict(mask=half), dict(mask=upper), dict(scale=0.0),
                dict(scale=float("inf")), dict(scale=3e38), dict(o=None), dict(o=FAKE + 2), dict(lens=FAKE + 2),
                dict(qs=(0, 0, 64)),  # as O's strides they let heads overlap
                dict(mask=fm._FmMask(FAKE + 4, FAKE, None, None, 1, 1))):
        assert call(lib, **bad) == fm.FM_ERR_INVALID_ARG, bad
    for bad in (dict(d=32), dict(H=3), dict(H=0), dict(N=0), dict(B=0), dict(max_pages=0),
                dict(mask=fm._FmMask(FAKE, FAKE, None, None, 3, 1)),
                dict(mask=fm._FmMask(FAKE, FAKE, None, None, 0, 1)), dict(B=1 << 20, N=1 << 12)):
        assert call(lib, **bad) == fm.FM_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 32), dict(ws_bytes=16)):
        assert call(lib, **bad) == fm.FM_ERR_WORKSPACE, bad
    assert fm.flashmask_cache_workspace_bytes(1, 4, 2, 1, 64, 4) > 0
    for bad in ((1, 4, 3, 1, 64, 4), (1, 4, 2, 1, 96, 4), (0, 4, 2, 1, 64, 4), (1, 4, 2, 1, 64, 0)):
        assert fm.flashmask_cache_workspace_bytes(*bad) == 0
