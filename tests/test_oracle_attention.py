"""The attention oracle against cases worked out by hand."""
import numpy as np

from oracle import attention as oa


def test_one_key_is_returned_and_no_key_is_nothing():
    v = np.arange(64.0).reshape(1, 1, 64)
    q = np.ones((2, 1, 64))
    out, lse, w, *_ = oa.attend(q, np.zeros((1, 1, 64)), v, 0.125, 0.0)
    assert np.array_equal(out[1, 0], v[0, 0]) and lse[1, 0] == 0.0 and w[0, 0] == 1.0
    assert not out[0].any() and lse[0, 0] == -np.inf


def test_two_keys_are_weighted_by_their_exponentials():
    k = np.zeros((2, 1, 64))
    k[0, 0, 3] = 1.0
    q = np.zeros((1, 2, 64))
    q[0, :, 3] = np.log(3.0)
    v = np.zeros((2, 1, 64))
    v[0, 0, 0], v[1, 0, 1] = 1.0, 1.0
    out, lse, w, *_ = oa.attend(q, k, v, 1.0, 0.0)
    assert np.allclose(out[0, 1, :2], [0.75, 0.25]) and np.allclose(lse, np.log(4.0)) and np.allclose(w[:, 0], [1.5, 0.5])


def test_eviction_by_hand():
    w = np.array([5.0, 1.0, 2.0, 2.0, 0.0, 9.0, 2.0, 0.0])
    at = np.arange(8)
    # 0, 5 and the first of the equal ones at 2 stay: 5 moves to the free place 1
    assert oa.evict(w, at, 3, 0, 0).tolist() == [0, 5, 2]
    # the last position stays whatever its weight
    assert oa.evict(w, at, 3, 1, 0).tolist() == [0, 5, 7]
    assert oa.evict(w, at[::-1].copy(), 2, 0, 1).tolist() == [5, 7]
    assert oa.evict(w, at, 8, 0, 0).tolist() == list(range(8))
    w[3] = np.nan
    assert oa.evict(w, at, 2, 0, 0).tolist() == [3, 5]
