"""Pins of the oracle's shared-prefix attention and eviction against facts fixed outside them.

- A shared prefix is the same as a copy of it in front of every sequence's own keys (attend_one).
- Sets of equal keys share the weight evenly; weights of a query sum to one per query head.
- The last query of several sees every key, an earlier one none behind its own; a query that sees
  nothing gives zeros.
- Query heads of one key head each read that head's columns.
- Eviction: hand-made cases for ties, the recent keys, NaN, and budgets that cut nothing.
"""
import numpy as np

from oracle import whisper_ref as R


def _kv(rng, n, heads):
    return rng.standard_normal((n, 64 * heads)), rng.standard_normal((n, 64 * heads))


def test_shared_prefix_is_a_copy_in_front_of_every_sequence():
    rng = np.random.default_rng(0)
    prefix = [_kv(rng, 5, 2), _kv(rng, 1, 2)]
    own = [_kv(rng, n, 2) for n in (3, 1, 4)]
    q = rng.standard_normal((3, 128))
    group_of = [0, 1, None]
    out, spread, wp, wo = R.prefix_attention(q, 1, 2, 2, prefix, group_of, own)
    for b in range(3):
        parts = ([prefix[group_of[b]]] if group_of[b] is not None else []) + [own[b]]
        k, v = (np.concatenate([x[j] for x in parts]) for j in range(2))
        np.testing.assert_allclose(out[b], R.attend_one(q[b], k, v, 2), rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(spread[b], R.attend_one(q[b], k, np.abs(v), 2), rtol=1e-12)
    total = wp[0].sum(1) + wp[1].sum(1) + sum(w.sum(1) for w in wo)
    np.testing.assert_allclose(total, 3.0)          # three queries of weight one in each head


def test_equal_keys_share_evenly():
    k = np.ones((4, 64))
    v = np.arange(4.0)[:, None] * np.ones((1, 64))
    out, _, wp, _ = R.prefix_attention(np.ones((2, 64)), 1, 1, 1, [(k, v)], [0, 0], [None, None])
    np.testing.assert_allclose(out, 1.5)
    np.testing.assert_allclose(wp[0], 0.5)          # two queries, a quarter each


def test_no_query_sees_a_key_behind_its_own():
    rng = np.random.default_rng(1)
    k, v = _kv(rng, 4, 1)
    q = rng.standard_normal((3, 64))
    out, _, _, wo = R.prefix_attention(q, 3, 1, 1, [], [None], [(k, v)])
    for i in range(3):
        np.testing.assert_allclose(out[i], R.attend_one(q[i], k[:2 + i], v[:2 + i], 1), rtol=1e-12)
    assert wo[0][0, 3] < 1.0                        # only the last query sees the last key
    short, _, _, _ = R.prefix_attention(q, 3, 1, 1, [], [None], [(k[:1], v[:1])])
    assert np.all(short[:2] == 0.0)                 # nothing to see
    np.testing.assert_allclose(short[2], v[0], rtol=1e-12)


def test_query_heads_read_their_key_head():
    rng = np.random.default_rng(2)
    k, v = _kv(rng, 6, 2)
    q = rng.standard_normal((1, 256))
    out, _, _, _ = R.prefix_attention(q, 1, 4, 2, [], [None], [(k, v)])
    for h in range(4):
        cols = slice(64 * (h // 2), 64 * (h // 2) + 64)
        np.testing.assert_allclose(out[0, 64 * h:64 * h + 64],
                                   R.attend_one(q[0, 64 * h:64 * h + 64], k[:, cols], v[:, cols], 1), rtol=1e-12)


def test_eviction_by_hand():
    keep = lambda w, m, r: R.cache_evict(np.array(w, np.float32), m, r).tolist()  # noqa: E731
    assert keep([5, 1, 3, 0, 0], 3, 1) == [0, 2, 4]
    assert keep([5, 1, 3, 0, 9], 3, 0) == [0, 2, 4]
    assert keep([1, 1, 1, 1], 2, 0) == [0, 1]                    # ties: the lowest index
    assert keep([0.0, -0.0, 0.0], 1, 0) == [0]                   # the zeros are equal
    assert keep([1, 2, 3], 3, 0) == [0, 1, 2] and keep([], 3, 1) == []
    assert keep([9, 8, 7, 0, 0], 2, 2) == [3, 4]                 # only recent keys
    assert keep([np.nan, -1, np.nan, 0], 2, 1) == [1, 3]         # NaN goes first
    assert keep([np.inf, 1, np.inf, 2], 2, 0) == [0, 2]
