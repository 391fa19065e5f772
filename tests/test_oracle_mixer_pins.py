"""The oracle of the token mixers beside causal attention, pinned against facts that do not come from it."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from oracle import mixers as X


def filled(rng, seq_len, heads=2, page=32, D=64):
    table, pages = C.page_table(rng, seq_len, page)
    c = O.Cache(pages, heads, page, D, rng)
    C.fill_cache(rng, c, table, seq_len)
    return c, table


def test_a_chain_as_a_tree_is_causal_attention():
    rng = np.random.default_rng(0)
    new, seq_len = [5, 0, 9], np.array([40, 7, 9])
    c, table = filled(rng, seq_len)
    start = C.ragged(new)
    q = rng.standard_normal((14, 4, 64)).astype(np.float32)
    words = np.concatenate([[(1 << (i + 1)) - 1 for i in range(n)] for n in new]).astype(np.uint64)[:, None]
    for window in (0, 12):
        want = O.attention(q, c, table, seq_len, start, 0.1, True, window)[0]
        got = X.attend(q, c, table, seq_len, start, 0.1,
                       lambda b, n, m, on: X.sees_tree(n, m, on, words[start[b]:start[b] + n], window))[0]
        assert np.allclose(got, want, rtol=1e-12, atol=1e-14)


def test_weights_of_a_row_sum_to_its_heads():
    rng = np.random.default_rng(1)
    seq_len, start = np.array([50]), np.array([0, 6])
    c, table = filled(rng, seq_len)
    q = rng.standard_normal((6, 4, 64)).astype(np.float32)
    _, _, reach, p = X.attend(q, c, table, seq_len, start, 0.1, lambda b, n, m, on: X.sees_position(n, m, on, True, 0))
    old = rng.random((1, 2, 64)).astype(np.float32)
    new, _ = X.weights(old, p, reach, 2, 2, seq_len, start, 2, 0.5)
    # two rows of two heads each give a token two probabilities a row; the older half fades, the call's own begin at 0
    assert np.allclose(new[0, :, :50].sum(axis=1), 0.5 * old[0, :, :44].sum(axis=1) + 4)
    assert np.array_equal(new[0, :, 50:], old[0, :, 50:])


def test_selection_by_hand():
    w = np.array([5, 1, 9, 9, 0, np.nan, 9, 2, 7, 3], np.float32)
    assert X.select(w, 10, 10, 0, 0).tolist() == list(range(10))
    assert X.select(w, 10, 2, 0, 0).tolist() == [2, 3]                       # of equal ones the lower
    assert X.select(w, 10, 5, 1, 2).tolist() == [0, 2, 3, 8, 9]
    assert X.select(w, 10, 9, 0, 0).tolist() == [0, 1, 2, 3, 4, 6, 7, 8, 9]  # the NaN goes first
    assert X.select(w, 10, 3, 1, 2).tolist() == [0, 8, 9]


@pytest.mark.parametrize("D", [64, 128])
def test_a_moved_token_reads_the_same(D):
    rng = np.random.default_rng(2)
    seq_len = np.array([60])
    c, table = filled(rng, seq_len, D=D)
    before = O.tokens_of(c, table[0], 60)
    X.move(c, table, seq_len, np.array([[[41, 43, 50]]]), np.array([3]), c, table, np.array([40]))
    after = O.tokens_of(c, table[0], 60)
    for x, y in zip(before[:2], after[:2]):
        assert np.array_equal(y[40:43], x[[41, 43, 50]])
        assert np.array_equal(y[43:], x[43:]) and np.array_equal(y[:40], x[:40])


def test_linear_attention_is_its_sum():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 7, 1, 8))
    v = rng.standard_normal((7, 2, 8))
    g, S0 = np.array([-0.3, 0.0]), rng.standard_normal((1, 2, 8, 8))
    o, S, _, _ = X.linear(q, k, v, g, S0, np.array([0, 7]), 0.5)
    for h in range(2):
        for i in range(7):
            want = np.exp(g[h] * (i + 1)) * q[i, 0] @ S0[0, h]
            want = want + sum(np.exp(g[h] * (i - j)) * (q[i, 0] @ k[j, 0]) * v[j, h] for j in range(i + 1))
            assert np.allclose(o[i, h], 0.5 * want)
        assert np.allclose(S[0, h], np.exp(7 * g[h]) * S0[0, h] + sum(np.exp(g[h] * (6 - j)) * np.outer(k[j, 0], v[j, h]) for j in range(7)))
