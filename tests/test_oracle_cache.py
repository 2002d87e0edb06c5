"""The plain forms in oracle.cache against other ways to the same values."""
import math

import numpy as np
import torch

from oracle import cache as C
from oracle import fp8 as F


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x, pos, f = rng.standard_normal((2, 3, 5, 10)), rng.integers(-99, 99, (2, 5)), rng.random(4)
    for inter in (False, True):
        y = C.rope(x, pos, f, inter, 1.5)
        first = np.arange(4) * (2 if inter else 1)
        second = first + (1 if inter else 4)
        z = (x[..., first] + 1j * x[..., second]) * 1.5 * np.exp(1j * pos[:, None, :, None] * f)
        assert np.allclose(y[..., first], z.real) and np.allclose(y[..., second], z.imag)
        assert np.array_equal(y[..., 8:], x[..., 8:])
        back = C.rope(y, pos, f, inter, 1 / 1.5, inverse=True)
        assert np.allclose(back, x)


def test_scale_exponent():
    for k in (-100, -3, 0, 7, 119):
        assert C.scale_exponent(448.0 * 2.0 ** k) == k
        assert C.scale_exponent(np.nextafter(448.0 * 2.0 ** k, np.inf)) == k + 1
        assert C.scale_exponent(224.0 * 2.0 ** k) == max(k - 1, -100)
    assert C.scale_exponent(0.0) == C.scale_exponent(1e-300) == -100


def test_append_in_pieces_equals_at_once_without_growth():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((1, 2, 90, 8)), rng.standard_normal((1, 2, 90, 8))
    k[:, :, (0, 64)] = v[:, :, (0, 64)] = 5.0  # the largest comes first in each page
    zero = np.zeros((3, 2, 64, 8)), np.ones((3, 2)), np.zeros((3, 2, 8, 64)), np.ones((3, 2))
    table = [[2, 0]]
    once = C.append(*zero, table, k, v, [0], None)
    parts = zero
    for s, e in ((0, 1), (1, 40), (40, 70), (70, 90)):
        parts = C.append(*parts, table, k[:, :, s:e], v[:, :, s:e], [s], None)
    for a, b in zip(once, parts):
        assert np.array_equal(a, b)
    got = (once[0] * once[1][..., None, None])[[2, 0]].transpose(1, 0, 2, 3).reshape(2, 128, 8)[:, :90]
    s = np.repeat(once[1][[2, 0]].T, 64, axis=1)[:, :90, None]
    assert np.array_equal(got, F.e4m3_round(k[0] / s) * s)


def test_attention_against_torch():
    gen = torch.Generator().manual_seed(0)
    B, H, Hk, N, d, n = 2, 4, 2, 3, 8, 100
    k8 = torch.randn((4, Hk, 64, d), generator=gen, dtype=torch.float64)
    v8 = torch.randn((4, Hk, d, 64), generator=gen, dtype=torch.float64)
    ks, vs = torch.rand((4, Hk), generator=gen).double(), torch.rand((4, Hk), generator=gen).double()
    q = torch.randn((B, H, N, d), generator=gen, dtype=torch.float64)
    table = [[3, 1], [0, 2]]
    o, lse, pv, _, _ = C.attend(q.numpy(), k8.numpy(), ks.numpy(), v8.numpy(), vs.numpy(), table, [n, n], None,
                             1 / math.sqrt(d))
    for b in range(B):
        k = (k8 * ks[..., None, None])[table[b]].transpose(0, 1).reshape(Hk, 128, d)[:, :n]
        v = (v8 * vs[..., None, None])[table[b]].permute(1, 0, 3, 2).reshape(Hk, 128, d)[:, :n]
        see = torch.arange(n) <= torch.arange(n - N, n)[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(
            q[b], k.repeat_interleave(2, 0), v.repeat_interleave(2, 0), attn_mask=see)
        assert np.allclose(o[b], want.numpy(), atol=1e-12)
        x = (q[b] @ k.repeat_interleave(2, 0).transpose(1, 2) / math.sqrt(d)).masked_fill(~see, -math.inf)
        assert np.allclose(lse[b], torch.logsumexp(x, -1).numpy(), atol=1e-12)
        assert (pv[b] >= np.abs(o[b]) - 1e-12).all()
