"""Norm with rotary positions and its gradients against the fp64 definition, the
gradients against differences, and the refusals (which need no GPU).

Tolerances, with u = 2^-24. Forward: the sum of squares adds at most 16 values a
thread, then over 32 lanes: 22 u relative, half of it in r, and rsqrtf 4 u; two products
2 u; the rotation as in test_gpu_rope: together below 2^-18 of mscale (|a| + |b|), of the
normed elements a, b of a pair, and the output's own rounding, half a step.
Backward: g carries 2^-20 of its pair, the sums 22 u of the sum of their terms'
magnitudes, r as above: below 2^-17 of r (|g w| + |x r| mean |g w x r|). dw: 2^-18 of
each term, and the chain of a sum: 16 heads a tile and at most 16 tiles here, then 5 + 8
+ 64 additions, 333 u < 2^-15 of the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm
from oracle import norm as O

from gpu_common import need_gpu

FAKE = 1 << 20
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
f64 = lambda t: None if t is None else t.double().cpu().numpy()


def close(got, want, tol, dtype):
    err = np.abs(f64(got) - want)
    tol = tol + np.abs(want) * HALF[dtype] * 1.01 + TINY[dtype] + 1e-37
    assert np.all(err <= tol), (err - tol).max()


def check_forward(y, x, w, pos, freqs, interleaved, mscale, eps):
    args = (f64(pos), f64(freqs), interleaved, mscale, eps)
    unit = O.forward(f64(x), f64(w), np.zeros_like(f64(pos)), [], eps=eps)
    mag = O.pair_magnitudes(unit, freqs.numel(), interleaved) * max(1.0, abs(mscale))
    close(y, O.forward(f64(x), f64(w), *args), mag * 2.0 ** -18, x.dtype)


def check_backward(dx, dw, dy, x, w, pos, freqs, interleaved, mscale, eps):
    args = (f64(pos), f64(freqs), interleaved, mscale, eps)
    want_x, want_w = O.backward(f64(dy), f64(x), f64(w), *args)
    g = O.pair_magnitudes(f64(dy), freqs.numel(), interleaved) * max(1.0, abs(mscale))
    r = 1.0 / np.sqrt(np.mean(f64(x) ** 2, -1, keepdims=True) + eps)
    u = np.abs(f64(x)) * r
    gw = g if w is None else g * np.abs(f64(w))
    close(dx, want_x, 2.0 ** -17 * r * (gw + u * np.mean(gw * u, -1, keepdims=True)), x.dtype)
    if w is None:
        assert dw is None
    else:
        assert dw.dtype == w.dtype and dw.shape == w.shape
        close(dw, want_w, (g * u).sum((0, 1, 2)) * (2.0 ** -18 + 2.0 ** -15), w.dtype)


def inputs(B, Hq, Hk, N, d, dtype, wdtype, seed=5):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda shape, dt: torch.randn(shape, generator=gen).to(dt).cuda()
    t = {"q": rn((B, Hq, N, d), dtype), "k": rn((B, Hk, N, d), dtype) * 3,
         "dq": rn((B, Hq, N, d), dtype), "dk": rn((B, Hk, N, d), dtype)}
    w = [None, None] if wdtype is None else [(1 + 0.3 * rn((d,), torch.float32)).to(wdtype) for _ in range(2)]
    pos = torch.randint(-(1 << 21), 1 << 21, (B, N), generator=gen).int().cuda()
    return t, w, pos


SHAPES = [(1, 1, 1, 1, 64, 64), (2, 8, 2, 33, 128, 128), (3, 5, 5, 17, 128, 64), (1, 3, 1, 300, 64, 54),
          (2, 7, 3, 9, 80, 20), (1, 2, 2, 5, 7, 6), (2, 4, 4, 3, 64, 0), (1, 2, 1, 40, 256, 256),
          (1, 2, 1, 11, 252, 120), (1, 17, 2, 6, 96, 96), (2, 1, 1, 3, 1, 0), (1, 2, 2, 70, 255, 254),
          (5, 40, 8, 1, 128, 128), (1, 3, 2, 4, 16, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", SHAPES)
def test_both_directions(dtype, interleaved, B, Hq, Hk, N, d, rot):
    fm = need_gpu()
    ws = fm.alloc_norm_workspace(d)
    ws.fill_(255)  # need not be zeroed
    freqs, _ = fm.rope_frequencies(rot, base=500000.0)
    for wdtype in (dtype, torch.float32, None):
        t, (qw, kw), pos = inputs(B, Hq, Hk, N, d, dtype, wdtype)
        how = dict(positions=pos, interleaved=interleaved, mscale=1.25, eps=1e-5)
        yq, yk = fm.flashmask_norm_rope(t["q"], t["k"], qw, kw, freqs, **how)
        check_forward(yq, t["q"], qw, pos, freqs, interleaved, 1.25, 1e-5)
        check_forward(yk, t["k"], kw, pos, freqs, interleaved, 1.25, 1e-5)
        got = fm.flashmask_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], qw, kw, freqs, ws, **how)
        check_backward(got[0], got[2], t["dq"], t["q"], qw, pos, freqs, interleaved, 1.25, 1e-5)
        check_backward(got[1], got[3], t["dk"], t["k"], kw, pos, freqs, interleaved, 1.25, 1e-5)
        # in place: forward over its input, gradients over dy and over x
        a, b = t["q"].clone(), t["k"].clone()
        fm.flashmask_norm_rope(a, b, qw, kw, freqs, out=(a, b), **how)
        assert torch.equal(a, yq) and torch.equal(b, yk)
        a, b = t["dq"].clone(), t["dk"].clone()
        fm.flashmask_norm_rope_bwd(a, b, t["q"], t["k"], qw, kw, freqs, ws, out=(a, b), **how)
        assert torch.equal(a, got[0]) and torch.equal(b, got[1])
        a, b = t["q"].clone(), t["k"].clone()
        again = fm.flashmask_norm_rope_bwd(t["dq"], t["dk"], a, b, qw, kw, freqs, ws, out=(a, b), **how)
        assert torch.equal(a, got[0]) and torch.equal(b, got[1])
        assert wdtype is None or (torch.equal(again[2], got[2]) and torch.equal(again[3], got[3]))
        # one tensor alone, default positions
        one = fm.flashmask_norm_rope(t["q"], None, qw, None, freqs, interleaved=interleaved)
        assert one[1] is None
        check_forward(one[0], t["q"], qw, torch.arange(N).expand(B, N), freqs, interleaved, 1.0, 1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tiles(dtype):
    # more tokens than the backward's CTAs take at once, heads that do not divide
    fm = need_gpu()
    B, Hq, Hk, N, d = 2, 19, 3, 5003, 64
    t, (qw, kw), pos = inputs(B, Hq, Hk, N, d, dtype, dtype)
    freqs, _ = fm.rope_frequencies(d)
    ws = fm.alloc_norm_workspace(d)
    how = dict(positions=pos[:1], eps=1e-6)
    yq, yk = fm.flashmask_norm_rope(t["q"], t["k"], qw, kw, freqs, **how)
    check_forward(yq, t["q"], qw, pos[:1].expand(B, N), freqs, False, 1.0, 1e-6)
    check_forward(yk, t["k"], kw, pos[:1].expand(B, N), freqs, False, 1.0, 1e-6)
    got = fm.flashmask_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], qw, kw, freqs, ws, **how)
    check_backward(got[0], got[2], t["dq"], t["q"], qw, pos[:1].expand(B, N), freqs, False, 1.0, 1e-6)
    check_backward(got[1], got[3], t["dk"], t["k"], kw, pos[:1].expand(B, N), freqs, False, 1.0, 1e-6)
    for _ in range(3):  # the same call, the same bits
        again = fm.flashmask_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], qw, kw, freqs, ws, **how)
        assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.gpu
def test_strides_and_broadcast():
    fm = need_gpu()
    B, H, N, d = 2, 4, 21, 128
    qkv = torch.randn((B, N, 3 * H * d), device="cuda").bfloat16()
    q, k = (qkv[..., i * H * d:(i + 1) * H * d].unflatten(2, (H, d)).transpose(1, 2) for i in (0, 1))
    t, (qw, kw), pos = inputs(B, H, H, N, d, torch.bfloat16, torch.float32)
    freqs, _ = fm.rope_frequencies(64)
    ws = fm.alloc_norm_workspace(d)
    want = fm.flashmask_norm_rope(q.contiguous(), k.contiguous(), qw, kw, freqs, positions=pos)
    got = fm.flashmask_norm_rope(q, k, qw, kw, freqs, positions=pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # odd offsets take the one-element path, which adds in another order
    buf = torch.zeros((B, H, N, d + 3), device="cuda").bfloat16()
    buf[..., 1:1 + d] = q
    out = torch.full((B, H, N, d + 3), 7.0, device="cuda").bfloat16()
    fm.flashmask_norm_rope(buf[..., 1:1 + d], None, qw, None, freqs, positions=pos, out=(out[..., 2:2 + d],))
    check_forward(out[..., 2:2 + d], q, qw, pos, freqs, False, 1.0, 1e-6)
    assert (out[..., :2] == 7).all() and (out[..., 2 + d:] == 7).all()
    # inputs that repeat: one head for all, one token for all
    x, g = t["q"][:, :1].expand(B, H, N, d), t["dq"][:, :, :1].expand(B, H, N, d)
    want = fm.flashmask_norm_rope_bwd(g.contiguous(), None, x.contiguous(), None, qw, None, freqs, ws, positions=pos)
    got = fm.flashmask_norm_rope_bwd(g, None, x, None, qw, None, freqs, ws, positions=pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    # in place inside the fused projection: V is left alone
    v = qkv[..., 2 * H * d:].clone()
    want = fm.flashmask_norm_rope(q, k, qw, kw, freqs, positions=pos)
    fm.flashmask_norm_rope(q, k, qw, kw, freqs, positions=pos, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[..., 2 * H * d:], v)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_heads(dtype):
    # zeros, tiny, huge (squares past fp32) and heads that are not finite, which spoil no other
    fm = need_gpu()
    d, N = 64, 8
    x = torch.randn((1, 2, N, d)).to(dtype)
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 1e-30
    x[0, 0, 2] *= 3e37
    x[0, 0, 3] *= 1e19
    x[0, 0, 4, 5] = float("inf")
    x[0, 0, 5, 6] = float("nan")
    x, w, g = x.cuda(), torch.rand(d).cuda() + 0.5, torch.randn((1, 2, N, d)).to(dtype).cuda()
    freqs, _ = fm.rope_frequencies(d)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    y, _ = fm.flashmask_norm_rope(x, None, w, None, freqs)
    dx, _, dw, _ = fm.flashmask_norm_rope_bwd(g, None, x, None, w, None, freqs, fm.alloc_norm_workspace(d))
    fine = [0, 1, 2, 3, 6, 7]
    for h, rows in ((0, fine), (1, list(range(N)))):
        pick = lambda t: t[:, h:h + 1, rows]
        check_forward(pick(y), pick(x), w, pos[:, rows], freqs, False, 1.0, 1e-6)
        got = pick(dx).contiguous()
        want, _ = O.backward(f64(pick(g)), f64(pick(x)), f64(w), f64(pos[:, rows]), f64(freqs))
        r = 1.0 / np.sqrt(np.mean(f64(pick(x)) ** 2, -1, keepdims=True) + 1e-6)
        u = np.abs(f64(pick(x))) * r
        gw = O.pair_magnitudes(f64(pick(g)), d // 2, False) * f64(w)
        close(got, want, 2.0 ** -17 * r * (gw + u * np.mean(gw * u, -1, keepdims=True)), dtype)
    assert torch.isnan(y[0, 0, 4]).any() and torch.isnan(y[0, 0, 5]).all()
    assert torch.isnan(dx[0, 0, 5]).all() and torch.isnan(dw).any()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 62])
def test_frequencies_of_all_sizes(d, interleaved):
    # the positions' turns are those of flashmask_rope for every frequency; one that is none
    # spoils its pair. In fp32 the two ways differ by the roundings of a turn's two products and
    # their sum, 4 u of the pair's magnitudes, and by r: which elements a thread adds up depends on
    # how many are turned, so each way's r is within 15 u of the exact one (half of 22 u, and 4 u)
    # and they within 30 u of one another: 34 u < 2^-18 in all
    fm = need_gpu()
    n, N = d // 2, 70
    gen = torch.Generator().manual_seed(d)
    f = 10.0 ** torch.linspace(-9, 38, n, dtype=torch.float64)
    f[1::3] *= -1
    f[2], f[3], f[4], f[5] = 0.0, 4.0, 2.0 ** 128, -5.0
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, N), generator=gen, dtype=torch.int64).int().cuda()
    x, g = (torch.randn((2, 3, N, d), generator=gen).cuda() for _ in range(2))
    w = (torch.rand(d, generator=gen) + 0.5).cuda()
    none = torch.empty(0, dtype=torch.float64, device="cuda")
    how = dict(positions=pos, interleaved=interleaved, mscale=1.5)
    flat, _ = fm.flashmask_norm_rope(x, None, w, None, none)
    for last in (None, float("nan"), float("inf"), 2.0 ** 129):
        if last is not None:
            f[7] = last
        freqs = f.cuda()
        want, _ = fm.flashmask_rope(flat, None, freqs, **how)
        got, _ = fm.flashmask_norm_rope(x, None, w, None, freqs, **how)
        spoilt = torch.isnan(want)
        assert torch.equal(torch.isnan(got), spoilt) and spoilt.any() == (last is not None)
        mag = torch.from_numpy(O.pair_magnitudes(f64(flat), n, interleaved)).cuda() * 1.5
        off = ((got.double() - want.double()).abs() / mag)[~spoilt].max()
        assert off <= 2.0 ** -18, off * 2.0 ** 24
        if last is None:
            turned, _ = fm.flashmask_rope_bwd(g, None, freqs, **how)
            ws = fm.alloc_norm_workspace(d)
            a = fm.flashmask_norm_rope_bwd(turned, None, x, None, w, None, none, ws)
            b = fm.flashmask_norm_rope_bwd(g, None, x, None, w, None, freqs, ws, **how)
            r = 1.0 / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
            u = x.double().abs() * r
            gw = torch.from_numpy(O.pair_magnitudes(f64(g), n, interleaved)).cuda() * 1.5 * w.double()
            bound = 2.0 ** -17 * r * (gw + u * (gw * u).mean(-1, keepdim=True))
            assert torch.all((a[0].double() - b[0].double()).abs() <= bound)
            assert torch.all((a[2].double() - b[2].double()).abs() <= 2.0 ** -17 * (gw / w.double() * u).sum((0, 1, 2)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 30)])
def test_weights_that_are_not_there(dtype, d):
    # none, and then no workspace either; Q's alone; K's alone
    fm = need_gpu()
    B, Hq, Hk, N = 2, 4, 2, 50
    t, w, _ = inputs(B, Hq, Hk, N, d, dtype, torch.float32)
    freqs, _ = fm.rope_frequencies(d)
    ws, ones = fm.alloc_norm_workspace(d), torch.ones(d, device="cuda")
    args = (t["dq"], t["dk"], t["q"], t["k"])
    for qw, kw in ((None, None), (w[0], None), (None, w[1])):
        full = [ones if x is None else x for x in (qw, kw)]
        for a, b in zip(fm.flashmask_norm_rope(t["q"], t["k"], qw, kw, freqs),
                        fm.flashmask_norm_rope(t["q"], t["k"], *full, freqs)):
            assert torch.equal(a, b)
        got = fm.flashmask_norm_rope_bwd(*args, qw, kw, freqs, None if qw is kw else ws)
        want = fm.flashmask_norm_rope_bwd(*args, *full, freqs, ws)
        for x, a, b in zip((1, 1, qw, kw), got, want):
            assert a is None if x is None else torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(interleaved):
    # central differences with step h in fp32: the error is h^2 / 6 of the third derivative
    # (below 8 |g| here, since r <= 4 and its derivatives are of the order of r^3) and 2^-19
    # of the loss's terms over h
    fm = need_gpu()
    gen = torch.Generator().manual_seed(1)
    x = (torch.randn((1, 2, 3, 8), generator=gen) + 1.0).cuda()
    g = torch.randn((1, 2, 3, 8), generator=gen).cuda()
    w = (1 + 0.3 * torch.randn(8, generator=gen)).cuda()
    freqs, _ = fm.rope_frequencies(6, base=100.0)
    pos = torch.tensor([[5, 0, -77]], dtype=torch.int32).cuda()
    kw = dict(positions=pos, interleaved=interleaved, mscale=1.5, eps=1e-2)
    dx, _, dw, _ = fm.flashmask_norm_rope_bwd(g, None, x, None, w, None, freqs, fm.alloc_norm_workspace(8), **kw)
    loss = lambda x, w: (fm.flashmask_norm_rope(x, None, w, None, freqs, **kw)[0].double() * g.double()).sum()
    y = fm.flashmask_norm_rope(x, None, w, None, freqs, **kw)[0]
    h = 2.0 ** -6
    noise = 2.0 ** -19 * float((y.abs() * g.abs()).sum()) * 1.5 / h
    for e in range(8):
        hi, lo = w.clone(), w.clone()
        hi[e] += h
        lo[e] -= h
        d = float(loss(x, hi) - loss(x, lo)) / float(hi[e] - lo[e])
        assert abs(d - float(dw[e])) <= noise
        for hd in range(2):
            for t in range(3):
                hi, lo = x.clone(), x.clone()
                hi[0, hd, t, e] += h
                lo[0, hd, t, e] -= h
                d = float(loss(hi, w) - loss(lo, w)) / float(hi[0, hd, t, e] - lo[0, hd, t, e])
                bend = h * h / 6 * 8 * 1.5 * float((g[0, hd, t].abs() * w.abs()).sum())
                assert abs(d - float(dx[0, hd, t, e])) <= noise + bend


@pytest.mark.gpu
def test_streams_and_graphs():
    fm = need_gpu()
    freqs, _ = fm.rope_frequencies(128)
    t, (qw, kw), pos = inputs(2, 8, 2, 50, 128, torch.bfloat16, torch.bfloat16)
    ws = fm.alloc_norm_workspace(128)
    args = (t["dq"], t["dk"], t["q"], t["k"], qw, kw, freqs, ws)
    fwd = (t["q"], t["k"], qw, kw, freqs)
    want, wanty = fm.flashmask_norm_rope_bwd(*args, positions=pos), fm.flashmask_norm_rope(*fwd, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fm.flashmask_norm_rope_bwd(*args, positions=pos, stream=s)
    goty = fm.flashmask_norm_rope(*fwd, positions=pos, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *goty), (*want, *wanty)))
    # two graphs that share the workspace
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fm.flashmask_norm_rope_bwd(*args, positions=pos))
        graphs.append(g)
    for k in range(2):
        t["q"].copy_(torch.randn_like(t["q"]))
        graphs[k].replay()
        want = fm.flashmask_norm_rope_bwd(*args, positions=pos)
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want))


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def call(lib, backward, x=FAKE, y=FAKE, dy=FAKE, w=FAKE, dw=FAKE, H=2, ys=(512, 256, 64), n=1, positions=None,
         freqs=FAKE, B=1, N=4, d=64, rot=64, dtype=fm.FM_BF16, wdtype=fm.FM_BF16, mscale=1.0, eps=1e-6, ws=FAKE,
         ws_bytes=1 << 30):
    t = (fm._FmNormHeads * 2)(*[fm._FmNormHeads(x, y, dy, w, dw, H, (0, 0, 0), ys, (0, 0, 0))] * 2)
    how = (t, n, positions, 0, freqs, B, N, d, rot, 0, dtype, wdtype, mscale, eps)
    return lib.flashmask_norm_rope_bwd(*how, ws, ws_bytes, None) if backward else \
        lib.flashmask_norm_rope(*how, None)


@pytest.mark.parametrize("backward", [False, True])
def test_refusals(lib, backward):
    bads = [dict(x=None), dict(y=None), dict(n=0), dict(n=3), dict(dtype=3), dict(dtype=-1), dict(freqs=None),
            dict(freqs=FAKE + 4), dict(positions=FAKE + 2), dict(x=FAKE + 1), dict(y=FAKE + 1), dict(w=FAKE + 1),
            dict(wdtype=fm.FM_F16), dict(mscale=float("nan")), dict(mscale=float("inf")), dict(eps=0.0),
            dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-31),
            dict(ys=(512, 0, 64)), dict(ys=(512, 256, 0)), dict(wdtype=fm.FM_F32, w=FAKE + 2)]
    if backward:
        bads += [dict(dy=None), dict(dy=FAKE + 1), dict(dw=FAKE + 1)]
    for bad in bads:
        assert call(lib, backward, **bad) == fm.FM_ERR_INVALID_ARG, bad
    for bad in (dict(B=0), dict(N=0), dict(H=0), dict(d=0), dict(d=257), dict(rot=66), dict(rot=-2), dict(rot=7),
                dict(H=70000), dict(B=1 << 16, N=1 << 16), dict(B=-1)):
        assert call(lib, backward, **bad) == fm.FM_ERR_UNSUPPORTED, bad
    if backward:
        for bad in (dict(ws=None), dict(ws=FAKE + 128), dict(ws_bytes=fm.flashmask_norm_workspace_bytes(64) - 1)):
            assert call(lib, backward, **bad) == fm.FM_ERR_WORKSPACE, bad
    assert fm.flashmask_norm_workspace_bytes(0) == 0 and fm.flashmask_norm_workspace_bytes(257) == 0


def test_binding_refusals():
    q, f = torch.zeros((1, 2, 4, 64)), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        fm.flashmask_norm_rope(q, None, None, None, f)  # not on a GPU
    with pytest.raises(ValueError):
        fm.flashmask_norm_rope(q.double(), None, None, None, f)
    with pytest.raises(fm.FlashMaskError):
        fm.alloc_norm_workspace(300)


@pytest.mark.gpu
def test_binding_refusals_on_tensors():
    fm = need_gpu()
    q, k = torch.zeros((2, 4, 3, 64), device="cuda"), torch.zeros((2, 2, 3, 64), device="cuda")
    w, f, ws = torch.ones(64, device="cuda"), torch.zeros(32, dtype=torch.float64, device="cuda"), \
        fm.alloc_norm_workspace(64)
    fm.flashmask_norm_rope_bwd(q, k, q, k, w, w, f, ws)
    for bad in (dict(q_weight=w[:32]), dict(q_weight=w.half()), dict(k_weight=w.double()),
                dict(q_weight=w.cpu()), dict(dk=None), dict(dq=q[:1]), dict(k=None), dict(freqs=f.float()),
                dict(ws=ws[:-1]), dict(ws=None), dict(positions=torch.zeros((2, 3), device="cuda")), dict(eps=0.0),
                dict(out=(q,)), dict(q_weight=torch.ones((64, 2), device="cuda")[:, 0])):
        args = dict(dq=q, dk=k, q=q, k=k, q_weight=w, k_weight=w, freqs=f, ws=ws)
        args.update(bad)
        with pytest.raises((ValueError, IndexError, fm.FlashMaskError)):
            fm.flashmask_norm_rope_bwd(**args)
    # mixed types of weights
    h = q.half()
    with pytest.raises(ValueError):
        fm.flashmask_norm_rope(h, h, w.half(), w, f)
