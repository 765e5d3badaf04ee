"""Closed forms that oracle/drafts.py and oracle/latent.py have to give."""
import numpy as np

from oracle import attention as plain
from oracle import drafts
from oracle import latent as ref
from test_oracle_attention_pins import cache


def test_masks_of_a_chain_are_the_causal_attention():
    rng = np.random.default_rng(1)
    k, v, table = cache(rng, 11)
    q = rng.standard_normal((5, 2, 8)).astype(np.float16)
    chain = np.array([1, 3, 7, 15, 31], dtype=np.int64)
    slopes = np.array([0.5, 0.1], dtype=np.float32)
    for window in (0, 3, 7):
        want = plain.attention(q, k, v, table, [0, 5], [11], 0.3, window=window, slopes=slopes)
        for masks in (chain, None):
            got = drafts.attention(q, k, v, table, [0, 5], [11], 0.3, masks, window=window, slopes=slopes)
            assert all(np.allclose(a, b) for a, b in zip(got[:2], want[:2])), (window, masks)


def test_a_tree_s_places_and_what_it_sees():
    # two siblings after the first token, a child of the second of them
    masks = np.array([0b0001, 0b0011, 0b0101, 0b1101], dtype=np.int64)
    seen, here, place = drafts.seen_and_places(masks, 4, 7)
    assert list(here) == [3, 4, 4, 5]
    assert list(place) == [0, 1, 2, 3, 4, 4, 5]
    assert np.array_equal(seen[:, :3], np.ones((4, 3), dtype=bool))
    assert np.array_equal(seen[:, 3:].astype(int), [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]])
    seen, _, _ = drafts.seen_and_places(masks, 4, 7, window=2)  # places above here - 2
    assert np.array_equal(seen.astype(int), [[0, 0, 1, 1, 0, 0, 0], [0, 0, 0, 1, 1, 0, 0], [0, 0, 0, 1, 0, 1, 0],
                                             [0, 0, 0, 0, 0, 1, 1]])


def test_masks_of_the_highest_bit_and_past_the_draft():
    named = drafts.bits(np.array([-2 ** 63] * 64, dtype=np.int64), 64)
    assert named[:, 63].all() and not named[:, :63].any()
    assert drafts.bits(np.array([0b110], dtype=np.int64), 1).tolist() == [[False]]
    # a token that nothing is named for keeps the first place
    _, here, _ = drafts.seen_and_places(np.zeros(2, dtype=np.int64), 2, 5)
    assert list(here) == [3, 3]


def test_siblings_do_not_see_each_other():
    rng = np.random.default_rng(2)
    k, v, table = cache(rng, 6)
    q = rng.standard_normal((3, 1, 8)).astype(np.float16)
    masks = np.array([1, 3, 5], dtype=np.int64)
    first, _, _ = drafts.attention(q, k, v, table, [0, 3], [6], 0.3, masks)
    p, o = plain.slot(table, 0, 4, 4, 5)  # drafted token 1
    k[p, :, o], v[p, :, :, o] = 9.0, 9.0
    again, _, _ = drafts.attention(q, k, v, table, [0, 3], [6], 0.3, masks)
    assert np.array_equal(first[[0, 2]], again[[0, 2]]) and not np.allclose(first[1], again[1])


def test_keep_moves_the_named_tokens():
    k, v, table = cache(np.random.default_rng(3), 12)
    got_k, got_v = drafts.keep(k, v, table, [3], [0, 3], [0, 2, 5])
    at = lambda j: (int(table[0, j // 4]), j % 4)  # noqa: E731
    for j in range(12):
        (p, o), (fp, fo) = at(j), at({4: 5, 5: 8}.get(j, j))
        assert np.array_equal(got_k[p, :, o], k[fp, :, fo]) and np.array_equal(got_v[p, :, :, o], v[fp, :, :, fo]), j
    rows = np.arange(5 * 4 * 2, dtype=np.float16).reshape(5, 4, 2)
    moved, none = drafts.keep(rows, None, table, [3], [0, 3], [0, 2, 5])
    assert none is None and np.array_equal(moved[0, :2], [rows[0, 1], rows[4, 0]]) and np.array_equal(moved[3], rows[3])


def test_latent_row():
    x = np.concatenate([np.full(128, -3.0), np.arange(64.0)])
    w = np.linspace(0.5, 2, 128)
    y = ref.row(x, 0, np.ones(32), 128, norm=w, eps=0.0)
    assert np.allclose(y[:128], -w) and np.array_equal(y[128:], x[128:])          # position 0 turns nothing
    y = ref.row(x, 1, np.full(32, np.pi / 2), 128, mscale=2.0)
    assert np.array_equal(y[:128], x[:128])
    assert np.allclose(y[128:160], -2 * x[160:]) and np.allclose(y[160:], 2 * x[128:160])  # a quarter turn, doubled
    assert np.array_equal(ref.turned(x[128:], 7, None), x[128:])


def latent_cache(rng):
    return rng.standard_normal((5, 4, 128 + ref.ROT)).astype(np.float16), np.array([[3, 0, 4, -1]], dtype=np.int32)


def test_latent_attention_averages_picks_and_skips():
    rows, table = latent_cache(np.random.default_rng(4))
    c, there = ref.rows_of(rows, table[0], 14)
    assert there.tolist() == [True] * 12 + [False] * 2
    q = np.zeros((2, 3, 128 + ref.ROT), dtype=np.float16)
    out, _, _ = ref.attention(q, rows, table, [0, 2], [7], 0.1)
    assert np.allclose(out[0], c[:6, :128].mean(0)) and np.allclose(out[1], c[:7, :128].mean(0))  # nothing asked: the mean
    q[1, 1] = (c[2] * 100).astype(np.float16)
    out, _, _ = ref.attention(q, rows, table, [0, 2], [7], 1.0)
    assert np.allclose(out[1, 1], c[2, :128])                                                     # its own row's by far
    out, mag, _ = ref.attention(q, rows, np.full((1, 4), -1, dtype=np.int32), [0, 2], [7], 1.0)
    assert not out.any() and not mag.any()                                                        # no pages: zeros
    masks = np.array([2, 1], dtype=np.int64)
    out, _, _ = ref.attention(q * 0, rows, table, [0, 2], [7], 1.0, masks)
    assert np.allclose(out[0], c[[0, 1, 2, 3, 4, 6], :128].mean(0)) and np.allclose(out[1], c[:6, :128].mean(0))


def test_both_forms_of_latent_attention_agree():
    rng = np.random.default_rng(5)
    rows, table = latent_cache(rng)
    heads, value, n = 2, 64, 9
    w = rng.standard_normal((heads * 2 * value, 128))
    keys, values = ref.expanded(rows, table, [n], w, heads)
    assert keys[0].shape == (n, heads, value + ref.ROT) and values[0].shape == (n, heads, value)
    split = w.reshape(heads, 2, value, 128)
    own = rng.standard_normal((1, heads, value + ref.ROT)) / 8
    absorbed = np.concatenate([np.einsum("thv,hvl->thl", own[:, :, :value], split[:, 0]), own[:, :, value:]], -1)
    mixed, _, _ = ref.attention(absorbed, rows, table, [0, 1], [n], 0.07)
    for h in range(heads):
        s = 0.07 * (keys[0][:, h] @ own[0, h])
        e = np.exp(s - s.max())
        assert np.allclose((e / e.sum()) @ values[0][:, h], split[h, 1] @ mixed[0, h])
