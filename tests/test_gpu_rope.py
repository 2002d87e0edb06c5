"""Rotary positions against the fp64 definition, the gradient against finite
differences of the forward, and the refusals (which need no GPU).

Tolerance: an output is one rounding of its type (half a step: bf16 2^-8, fp16
2^-11, fp32 2^-24 of the value) plus the fp32 work before it: the angle in half
turns is rounded to 24 bits (pi 2^-24 rad), sincospif is good to 2 ulp (2^-22),
two products and a sum add 3 * 2^-24: together below 2^-20 of mscale (|x| +
|y|). fp16 results below 2^-14 have an absolute step of 2^-24."""
import ctypes

import numpy as np
import pytest
import torch

from mask_aware_exact_gb300 import flashmask as fm
from oracle import cache as C

from gpu_common import need_gpu

FAKE = 1 << 20
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def check(y, x, positions, freqs, interleaved, mscale, inverse, dtype):
    f = lambda t: t.double().cpu().numpy()
    ref = C.rope(f(x), f(positions), f(freqs), interleaved, mscale, inverse)
    n = freqs.numel()
    mag = np.abs(f(x))
    pair = mag.copy()
    first = 2 * np.arange(n) if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    pair[..., first] = pair[..., second] = mag[..., first] + mag[..., second]
    tol = abs(mscale) * pair * 2.0 ** -20 + np.abs(ref) * HALF[dtype] * 1.01 + 2.0 ** -25
    tol[..., 2 * n:] = 0.0  # copied
    err = np.abs(f(y) - ref)
    assert np.all(err <= tol), (err - tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", [(1, 1, 1, 1, 64, 64), (2, 8, 2, 33, 128, 128),
                                             (3, 5, 5, 17, 128, 64), (1, 3, 1, 300, 64, 54),
                                             (2, 7, 3, 9, 80, 20), (1, 2, 2, 5, 7, 6),
                                             (2, 4, 4, 3, 64, 0)])
def test_rotation(dtype, interleaved, inverse, B, Hq, Hk, N, d, rot):
    fm = need_gpu()
    gen = torch.Generator().manual_seed(7)
    q = torch.randn((B, Hq, N, d), generator=gen).to(dtype).cuda()
    k = (torch.randn((B, Hk, N, d), generator=gen) * 3).to(dtype).cuda()
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (B, N), generator=gen).int().cuda()
    freqs, _ = fm.rope_frequencies(rot, base=500000.0)
    call = fm.flashmask_rope_bwd if inverse else fm.flashmask_rope
    # the positions' own products must be exact: the definition in fp64 has 53
    # bits, so far positions are compared at magnitudes below 2^22
    pos = pos % (1 << 22) - (1 << 21)
    yq, yk = call(q, k, freqs, positions=pos, interleaved=interleaved, mscale=1.25)
    check(yq, q, pos, freqs, interleaved, 1.25, inverse, dtype)
    check(yk, k, pos, freqs, interleaved, 1.25, inverse, dtype)
    # one tensor alone, default positions
    y1, none = call(q, None, freqs, interleaved=interleaved)
    assert none is None
    check(y1, q, torch.arange(N).expand(B, N), freqs, interleaved, 1.0, inverse, dtype)
    # in place
    call(q2 := q.clone(), k2 := k.clone(), freqs, positions=pos, interleaved=interleaved, mscale=1.25,
         out=(q2, k2))
    assert torch.equal(q2, yq) and torch.equal(k2, yk)


@pytest.mark.gpu
@pytest.mark.parametrize("scaling", ["linear", "parts"])
def test_far_positions_and_scaling(scaling):
    # 2^31 - 1 positions on: the angle is exact modulo a turn
    fm = need_gpu()
    freqs, mscale = fm.rope_frequencies(64, 10000.0, scaling, 8.0, 4096)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 1000003, 0]], dtype=torch.int32).cuda()
    x = torch.zeros((1, 1, 4, 64), device="cuda")
    x[..., :32] = 1.0  # (cos, sin) of every pair
    y, _ = fm.flashmask_rope(x, None, freqs, positions=pos, mscale=mscale)
    from fractions import Fraction
    import math
    # 2 pi to 120 bits: position times frequency exactly, then modulo a turn
    two_pi = Fraction(math.pi) * 2 + Fraction(2 * 1.2246467991473532e-16)
    for t in range(4):
        for i in range(32):
            a = Fraction(int(pos[0, t])) * Fraction(float(freqs[i])) % two_pi
            for got, want in ((y[0, 0, t, i], math.cos(a)), (y[0, 0, t, 32 + i], math.sin(a))):
                assert abs(float(got) - mscale * want) <= mscale * 2.0 ** -20


@pytest.mark.gpu
def test_strided_and_shared_positions():
    fm = need_gpu()
    B, H, N, d = 2, 4, 21, 128
    qkv = torch.randn((B, N, 3 * H * d), device="cuda").bfloat16()
    q, k = (qkv[..., i * H * d:(i + 1) * H * d].unflatten(2, (H, d)).transpose(1, 2) for i in (0, 1))
    freqs, _ = fm.rope_frequencies(128)
    pos = torch.randint(0, 9999, (1, N), device="cuda", dtype=torch.int32)
    yq, yk = fm.flashmask_rope(q, k, freqs, positions=pos)
    check(yq, q, pos.expand(B, N), freqs, False, 1.0, False, torch.bfloat16)
    # into a strided place, odd offsets (the one-element path)
    buf = torch.zeros((B, H, N, d + 3), device="cuda").bfloat16()
    fm.flashmask_rope(q, None, freqs, positions=pos, out=(buf[..., 1:1 + d],))
    assert torch.equal(buf[..., 1:1 + d], yq)
    assert (buf[..., 0] == 0).all() and (buf[..., 1 + d:] == 0).all()
    # in place inside the fused projection: V is left alone
    v = qkv[..., 2 * H * d:].clone()
    fm.flashmask_rope(q, k, freqs, positions=pos, out=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[..., 2 * H * d:], v)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    # the map is linear, so central differences with a large step are exact up
    # to fp32 rounding: |dL/dx - difference| <= 2^-18 sum |g| |R|
    fm = need_gpu()
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((1, 2, 3, 8), generator=gen).cuda()
    g = torch.randn((1, 2, 3, 8), generator=gen).cuda()
    freqs, _ = fm.rope_frequencies(6, base=100.0)
    pos = torch.tensor([[5, 0, -77]], dtype=torch.int32).cuda()
    kw = dict(positions=pos, interleaved=interleaved, mscale=1.5)
    dx, _ = fm.flashmask_rope_bwd(g, None, freqs, **kw)
    for h in range(2):
        for t in range(3):
            for e in range(8):
                hi, lo = x.clone(), x.clone()
                hi[0, h, t, e] += 1.0
                lo[0, h, t, e] -= 1.0
                f = lambda z: (fm.flashmask_rope(z, None, freqs, **kw)[0].double() * g.double()).sum()
                d = float(f(hi) - f(lo)) / float(hi[0, h, t, e] - lo[0, h, t, e])
                assert abs(d - float(dx[0, h, t, e])) <= 2.0 ** -18 * float(g.abs().sum()) * 1.5


@pytest.mark.gpu
def test_nan_frequency_stays_in_its_pair():
    fm = need_gpu()
    freqs, _ = fm.rope_frequencies(64)
    freqs[3] = float("inf")
    x = torch.randn((1, 1, 4, 64), device="cuda")
    y, _ = fm.flashmask_rope(x, None, freqs)
    bad = torch.isnan(y[0, 0]).any(0).nonzero()[:, 0].tolist()
    assert bad == [3, 35]


@pytest.mark.gpu
def test_side_stream_and_graph():
    fm = need_gpu()
    freqs, _ = fm.rope_frequencies(128)
    q, k = torch.randn((2, 8, 50, 128), device="cuda").bfloat16(), torch.randn((2, 2, 50, 128), device="cuda").bfloat16()
    want = fm.flashmask_rope(q, k, freqs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fm.flashmask_rope(q, k, freqs, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fm.flashmask_rope(q, k, freqs)
    q.copy_(torch.randn_like(q))
    g.replay()
    want = fm.flashmask_rope(q, k, freqs)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.fixture(scope="module")
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def call(lib, x=FAKE, y=FAKE, H=2, ys=(512, 256, 64), n=1, positions=None, freqs=FAKE, B=1, N=4, d=64, rot=64,
         dtype=fm.FM_BF16, mscale=1.0):
    t = (fm._FmHeads * 2)(*[fm._FmHeads(x, y, H, (0, 0, 0), ys)] * 2)
    return lib.flashmask_rope(t, n, positions, 0, freqs, B, N, d, rot, 0, dtype, mscale, 0, None)


def test_refusals(lib):
    for bad in (dict(x=None), dict(y=None), dict(n=0), dict(n=3), dict(dtype=3), dict(freqs=None),
                dict(freqs=FAKE + 4), dict(positions=FAKE + 2), dict(x=FAKE + 1),
                dict(mscale=float("nan")), dict(ys=(512, 0, 64)), dict(ys=(512, 256, 0))):
        assert call(lib, **bad) == fm.FM_ERR_INVALID_ARG, bad
    for bad in (dict(B=0), dict(N=0), dict(H=0), dict(d=0), dict(rot=66), dict(rot=-2), dict(rot=7),
                dict(H=70000), dict(B=1 << 16, N=1 << 16)):
        assert call(lib, **bad) == fm.FM_ERR_UNSUPPORTED, bad
    assert lib.flashmask_rope(None, 1, None, 0, FAKE, 1, 1, 64, 64, 0, 0, 1.0, 0, None) == \
        fm.FM_ERR_INVALID_ARG


def test_binding_refusals():
    q = torch.zeros((1, 2, 4, 64))
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        fm.flashmask_rope(q, None, f)  # not on a GPU
    with pytest.raises(ValueError):
        fm.flashmask_rope(q.double(), None, f)
    for kw in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=4, base=-1.0),
               dict(rot_dim=4, scaling="other"), dict(rot_dim=4, scaling="parts", fast=1, slow=1)):
        with pytest.raises(ValueError):
            fm.rope_frequencies(**kw, device="cpu")


def test_frequencies():
    f, c = fm.rope_frequencies(8, 10000.0, device="cpu")
    assert c == 1.0 and np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    lin, _ = fm.rope_frequencies(8, 10000.0, "linear", 4.0, device="cpu")
    assert np.allclose(lin.numpy(), f.numpy() / 4, rtol=1e-15)
    part, c = fm.rope_frequencies(8, 10000.0, "parts", 4.0, original=1000, device="cpu")
    # turns within 1000 positions: 159.2 (kept), 15.92 (mixed), 1.592 (mixed), 0.159 (divided)
    g = [(1000 * x / (2 * np.pi) - 1) / 31 for x in f.numpy()[1:3]]
    want = [1.0, g[0] * 0.1 + (1 - g[0]) * 0.025, g[1] * 0.01 + (1 - g[1]) * 0.0025, 0.00025]
    assert np.allclose(part.numpy(), want, rtol=1e-12) and abs(c - (0.1 * np.log(4.0) + 1)) < 1e-15
    assert fm.rope_frequencies(0, device="cpu")[0].numel() == 0
