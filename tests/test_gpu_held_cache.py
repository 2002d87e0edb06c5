"""The calls around a cache that is held to a size, in turn as a server makes them:
normed rotary positions, append, attention, the keys' weights, eviction. A second copy of
the sequence is kept in fp64 beside it: the tokens that the cache should hold, with the
values that it holds for them."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C
from oracle import evict as E
from oracle import norm as O

from cache_common import PAGE, attention_bounds, cache_arrays, random_table
from gpu_common import need_gpu

f64 = lambda t: t.double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("d,H,Hk", [(128, 8, 2), (64, 4, 4)])
def test_a_served_sequence(d, H, Hk):
    fm = need_gpu()
    B, prompt, window, steps, size = 2, [300, 211], 32, 6, 128
    gen = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(s, generator=gen)
    freqs, mscale = fm.rope_frequencies(d)
    qw, kw = (1 + 0.2 * rn(d)).cuda(), (1 + 0.2 * rn(d)).cuda()
    table = random_table([n + steps for n in prompt], 6, gen)
    cache = fm.KVCache.empty(int(sum(-(-(n + steps) // PAGE) for n in prompt)), Hk, d)
    weights = torch.full((cache.k8.shape[0], Hk, PAGE), 9.0, device="cuda")  # of nothing yet
    N = max(prompt)
    ws = fm.alloc_cache_workspace(B, H, Hk, N, d, 6)
    wws, ews = fm.alloc_cache_weights_workspace(B, H, Hk, N, d, 6), fm.alloc_cache_evict_workspace(B, Hk, 6)
    held = torch.zeros(B, dtype=torch.int32, device="cuda")
    position = torch.zeros(B, dtype=torch.int32, device="cuda")

    def turn(count, rows, start, appended=True):
        """One pass over `rows` tokens a sequence, count of them real."""
        nonlocal held, position
        n = torch.tensor(count, dtype=torch.int32, device="cuda")
        q, k, v = (rn(B, h, rows, d).bfloat16().cuda() for h in (H, Hk, Hk))
        pos = position[:, None] + torch.arange(rows, dtype=torch.int32, device="cuda")
        pos = pos.int().contiguous()
        qr, kr = fm.flashmask_norm_rope(q, k, qw, kw, freqs, positions=pos, mscale=mscale)
        for y, x, w in ((qr, q, qw), (kr, k, kw)):
            want = O.forward(f64(x), f64(w), f64(pos), f64(freqs), False, mscale, 1e-6)
            mag = O.pair_magnitudes(O.forward(f64(x), f64(w), np.zeros((B, rows)), []), d // 2, False)
            assert np.all(np.abs(f64(y) - want) <= mag * 2.0 ** -18 + np.abs(want) * 2.0 ** -8 * 1.01)
        fm.flashmask_cache_append(cache, table, kr, v, held, ws, count=n)
        held, position = held + n, position + n
        o, lse = fm.flashmask_fwd_cache(qr, cache, table, held, ws, q_lens=n)
        # the last rows of each sequence weigh its keys
        last = min(rows, window)
        ql = n.clamp(max=last)
        first = (n - ql).long()
        take = (first[:, None] + torch.arange(last, device="cuda")).clamp(max=rows - 1)
        qr2 = torch.gather(qr, 2, take[:, None, :, None].expand(B, H, last, d))
        lse2 = torch.gather(lse, 2, take[:, None].expand(B, H, last)).contiguous()
        old = f64(weights)
        fm.flashmask_cache_weights(qr2, cache, table, held, lse2, weights, wws, q_lens=ql, start=start)
        arrays = cache_arrays(cache)
        args = (table.cpu().numpy(), held.tolist())
        ref = C.attend(f64(qr), *arrays, *args, count, 1 / math.sqrt(d))
        tol_o, tol_l = attention_bounds(ref, int(held.max()))
        for b in range(B):
            rows_b = slice(0, count[b])
            assert np.all(np.abs(f64(o)[b, :, rows_b] - ref[0][b, :, rows_b]) <= tol_o[b, :, rows_b])
        want, tol = E.weigh(f64(qr2), arrays[0], arrays[1], *args, ql.tolist(), f64(lse2), old,
                            None if start is None else start.tolist(), 1 / math.sqrt(d))
        assert np.all(np.abs(f64(weights) - want) <= tol + 1e-30)

    def evict():
        nonlocal held
        before = cache_arrays(cache) + (f64(weights),)
        lens = held.tolist()
        want = E.evict(*before, table.cpu().numpy(), lens, [size] * B, 4, 16)
        held = fm.flashmask_cache_evict(cache, table, held, weights, size, ews, sink=4, recent=16)
        assert held.tolist() == [min(n, size) for n in lens]
        for x, y in zip(cache_arrays(cache) + (f64(weights),), want[:5]):
            np.testing.assert_array_equal(x, y)

    turn(prompt, N, torch.zeros(B, dtype=torch.int32, device="cuda"))
    evict()
    for step in range(steps):
        turn([1, 1], 1, None)
        if step % 3 == 2:
            evict()
    for w in (ws, wws, ews):
        assert fm.flashmask_check_status(w) == (fm.FM_OK, 0)


@pytest.mark.gpu
def test_a_training_step_with_normed_heads():
    # norm and rotation, attention, and the gradients back through both: against the chain
    # of the two oracles' gradients at the kernels' own intermediate values
    fm = need_gpu()
    from mask_aware_exact_gb300 import workloads as W
    B, H, N, d = 1, 2, 200, 64
    q, k, v, do = W.make_qkv(B, H, N, d, 4)
    mask = fm.DeviceMask.from_spec(W.causal_bounds(B, 1, N))
    freqs, _ = fm.rope_frequencies(d)
    w = [(1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(i))).cuda() for i in (0, 1)]
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    ws, nws = fm.alloc_workspace(B, H, 1, N, d), fm.alloc_norm_workspace(d)
    qr, kr = fm.flashmask_norm_rope(q, k, *w, freqs)
    o, lse = fm.flashmask_fwd(qr, kr, v, mask, ws)
    dqr, dkr, _ = fm.flashmask_bwd(qr, kr, v, o, lse, do, mask, ws, ws_classified=True)
    dq, dk, dqw, dkw = fm.flashmask_norm_rope_bwd(dqr, dkr, q, k, *w, freqs, nws)
    pos = np.arange(N)[None].repeat(B, 0)
    for got, gw, g, x, wt in ((dq, dqw, dqr, q, w[0]), (dk, dkw, dkr, k, w[1])):
        dx, dw = O.backward(f64(g), f64(x), f64(wt), pos, f64(freqs))
        assert np.linalg.norm(f64(got) - dx) <= 2.0 ** -8 * np.linalg.norm(dx)
        terms = (np.abs(O.pair_magnitudes(f64(g), d // 2, False)) * np.abs(f64(x)) /
                 np.sqrt(np.mean(f64(x) ** 2, -1, keepdims=True))).sum((0, 1, 2))
        assert np.all(np.abs(f64(gw) - dw) <= terms * 2.0 ** -14)
    assert fm.flashmask_check_status(ws) == (fm.FM_OK, 0)


@pytest.mark.gpu
def test_two_servers_at_once():
    # the same calls on two streams, each with workspaces of its own, give what they give
    # one after the other
    fm = need_gpu()
    H, Hk, d, N, lens, keep = 8, 2, 128, 40, [3000, 1000, 77], 500

    def server(seed):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=gen)
        table = random_table(lens, 47, gen)
        out = torch.arange(3 * 8, dtype=torch.int32).view(3, 8) + 65
        cache = fm.KVCache.empty(65 + 24, Hk, d)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        k, v = (rn(3, Hk, max(lens), d).bfloat16().cuda() for _ in range(2))
        ws = fm.alloc_cache_workspace(3, H, Hk, N, d, 47)
        fm.flashmask_cache_append(cache, table, k, v, ints([0] * 3), ws, count=ints(lens))
        return dict(q=rn(3, H, N, d).bfloat16().cuda(), qw=rn(d).cuda(), cache=cache, table=table, out=out.cuda(),
                    lens=ints(lens), ws=ws, wws=fm.alloc_cache_weights_workspace(3, H, Hk, N, d, 47),
                    ews=fm.alloc_cache_evict_workspace(3, Hk, 47), nws=fm.alloc_norm_workspace(d))

    freqs, mscale = fm.rope_frequencies(d)

    def turn(s):
        q, _ = fm.flashmask_norm_rope(s["q"], None, s["qw"], None, freqs, mscale=mscale)
        o, lse = fm.flashmask_fwd_cache(q, s["cache"], s["table"], s["lens"], s["ws"])
        w = torch.zeros((89, Hk, PAGE), device="cuda")
        start = torch.zeros(3, dtype=torch.int32, device="cuda")
        fm.flashmask_cache_weights(q, s["cache"], s["table"], s["lens"], lse, w, s["wws"], start=start)
        new = fm.flashmask_cache_evict(s["cache"], s["table"], s["lens"], w, keep, s["ews"], sink=4, recent=16,
                                       out_table=s["out"])
        dq, _, dw, _ = fm.flashmask_norm_rope_bwd(o, None, s["q"], None, s["qw"], None, freqs, s["nws"], mscale=mscale)
        codes = [t[s["out"].flatten().long()].clone().view(torch.uint8) for t in (*s["cache"].tensors, w)]
        return [q, o, lse, w, new, dq, dw, *codes]

    servers = [server(1), server(2)]
    want = [turn(s) for s in servers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in servers]
    got = [[], []]
    for _ in range(6):
        for i, (s, stream) in enumerate(zip(servers, streams)):
            with torch.cuda.stream(stream):
                got[i].append(turn(s))
    torch.cuda.synchronize()
    for i, s in enumerate(servers):
        for x in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(x, want[i]))
        for name in ("ws", "wws", "ews"):
            assert fm.flashmask_check_status(s[name]) == (fm.FM_OK, 0)
