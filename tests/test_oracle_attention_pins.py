"""Closed forms that oracle/attention.py has to give."""
import numpy as np

from oracle import attention as ref


def test_rotation_keeps_lengths_and_turns_by_the_angle():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(8)
    freq = np.array([np.pi / 2, 0.0, 0.1])
    for inter in (False, True):
        y = ref.rotated(x, 1, freq, 6, inter)
        lo, hi = (0, 1) if inter else (0, 3)
        assert np.allclose([y[lo], y[hi]], [-x[hi], x[lo]])        # a quarter turn
        assert np.array_equal(y[6:], x[6:])                        # the rest passes
        assert np.isclose(np.linalg.norm(y), np.linalg.norm(x))
        assert np.allclose(ref.rotated(x, 0, freq, 6, inter), x)   # position 0 turns nothing
    # scores depend on the distance only
    q, k = rng.standard_normal(8), rng.standard_normal(8)
    a = ref.rotated(q, 9, freq, 6) @ ref.rotated(k, 4, freq, 6)
    b = ref.rotated(q, 105, freq, 6) @ ref.rotated(k, 100, freq, 6)
    assert np.isclose(a, b)


def test_norm_gives_unit_mean_square():
    y = ref.rotated(np.arange(1.0, 9.0), 0, [], 0, weight=np.ones(8), eps=0.0)
    assert np.isclose(np.mean(y * y), 1.0)


def cache(rng, n, page=4, dim=8):
    k = rng.standard_normal((5, 1, page, dim)).astype(np.float16)
    v = rng.standard_normal((5, 1, dim, page)).astype(np.float16)
    return k, v, np.array([[3, 0, 4, -1]], dtype=np.int32)


def test_equal_keys_average_the_values():
    k, v, table = cache(np.random.default_rng(1), 10)
    k[:] = 1
    q = np.ones((10, 1, 8), dtype=np.float16)
    out, _, _ = ref.attention(q, k, v, table, [0, 10], [10], 0.3)
    rows = np.stack([v[table[0, j // 4], 0, :, j % 4] for j in range(10)]).astype(np.float64)
    for t in range(10):
        assert np.allclose(out[t, 0], rows[:t + 1].mean(0))
    out, _, _ = ref.attention(q, k, v, table, [0, 10], [10], 0.3, window=3)
    assert np.allclose(out[9, 0], rows[7:10].mean(0))
    out, _, _ = ref.attention(q, k, v, table, [0, 10], [10], 0.3, prefix=[6])
    assert np.allclose(out[2, 0], rows[:6].mean(0))
    assert np.allclose(out[8, 0], rows[:9].mean(0))


def test_absent_pages_and_empty_rows():
    k, v, table = cache(np.random.default_rng(2), 14)
    q = np.ones((1, 1, 8), dtype=np.float16)
    with_page, _, _ = ref.attention(q, k, v, table, [0, 1], [14], 0.3)   # positions 12, 13 have no page
    without, _, _ = ref.attention(q, k, v, table, [0, 1], [12], 0.3)
    assert np.allclose(with_page, without)
    out, _, _ = ref.attention(q, k, v, table, [0, 1], [0], 0.3)
    assert not out.any()


def test_a_large_score_takes_all_and_a_cap_limits_it():
    k, v, table = cache(np.random.default_rng(3), 8)
    k[:] = 0
    k[3, 0, 2] = 1
    q = np.full((1, 1, 8), 100, dtype=np.float16)
    out, _, _ = ref.attention(q, k, v, table, [0, 1], [8], 1.0)
    assert np.allclose(out[0, 0], v[3, 0, :, 2])
    w = ref.weights(q[0, 0], k[3, 0].astype(float), 3, np.ones(4, bool), 1.0, softcap=2.0)
    assert np.isclose(w[2] / w[0], np.exp(2.0))
    w = ref.weights(q[0, 0] * 0, k[3, 0].astype(float), 3, np.ones(4, bool), 1.0, slope=0.5)
    assert np.allclose(w[1:] / w[:-1], np.exp(0.5))
