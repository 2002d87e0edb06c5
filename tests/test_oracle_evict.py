"""The oracles of the keys' weights and of eviction on cases worked by hand."""
import numpy as np

from oracle import evict as E


def test_kept():
    nan = float("nan")
    assert E.kept([5, 1, 3, 2, 4], 5, 3, 0, 0) == [0, 2, 4]
    assert E.kept([5, 1, 3, 2, 4], 5, 3, 0, 1) == [0, 2, 4]
    assert E.kept([0, 1, 3, 2, 0], 5, 3, 1, 1) == [0, 2, 4]
    assert E.kept([1, 1, 1, 1], 4, 2, 0, 0) == [0, 1]        # equal: the lower position
    assert E.kept([nan, -1, 0.0, -0.0], 4, 2, 0, 0) == [2, 3]
    assert E.kept([nan, -np.inf], 2, 1, 0, 0) == [1]
    assert E.kept([1, 2, 3], 3, 9, 1, 1) == [0, 1, 2]
    assert E.kept([1, 2, 3], 3, 2, 5, 5) == [0, 1]           # the first count before the last
    assert E.kept([1, 2, 3], 3, 0, 5, 5) == []


def test_weigh_by_hand():
    # two keys, one query at the second: scores 0 and ln 3, so the weights are 1/4 and 3/4
    d = 64
    k8 = np.zeros((1, 1, 64, d))
    k8[0, 0, 1, 0] = np.log(3.0)
    q = np.zeros((1, 1, 1, d))
    q[..., 0] = 1.0
    lse = np.array([[[np.log(4.0)]]])
    old = np.full((1, 1, 64), 2.0)
    w, _ = E.weigh(q, k8, np.ones((1, 1)), [[0]], [2], None, lse, old, None, 1.0)
    assert np.allclose(w[0, 0, :3], [2.25, 0.75, 2.0])  # key 0 is old, key 1 the query's own
    w, _ = E.weigh(q, k8, np.ones((1, 1)), [[0]], [2], None, lse, old, [0], 1.0)
    assert np.allclose(w[0, 0, :2], [0.25, 0.75])


def test_evict_by_hand():
    d = 64
    k8, v8 = np.zeros((2, 1, 64, d)), np.zeros((2, 1, d, 64))
    k8[0, 0, :, 0] = np.arange(64) % 8
    k8[1, 0, 5, 0] = 448.0
    v8[0, 0, 0, :] = np.arange(64) % 4
    w = np.zeros((2, 1, 64))
    w[0, 0, [3, 9]] = 1.0, 2.0
    w[1, 0, 5] = 5.0
    out = E.evict(k8, np.ones((2, 1)), v8, np.ones((2, 1)), w, [[0, 1]], [70], [3], 0, 0)
    assert out[5] == [[[3, 9, 69]]]
    assert out[0][0, 0, :4, 0].tolist() == [3.0, 1.0, 448.0, 0.0] and out[1][0, 0] == 1.0
    # V's largest is 3: 3 / 448 <= 2^-7, and codes are values over 2^-7
    assert out[3][0, 0] == 2.0 ** -7 and out[2][0, 0, 0, :3].tolist() == [384.0, 128.0, 0.0]
    assert out[4][0, 0, :4].tolist() == [1.0, 2.0, 5.0, 0.0]
