"""The oracle of the calls between a layer's linears, pinned against facts that do not come from it."""
import numpy as np
import pytest

from oracle import layer as O


def test_e2m1_levels_ties_and_signs():
    # every level keeps its code; the middle of two levels goes to the even index; beyond 6 stays 6
    assert O.e2m1_codes(np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 7, 1e9])).tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 7, 7]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert O.e2m1_codes(mids).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert O.e2m1_codes(np.nextafter(mids, 10)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert O.e2m1_codes(np.nextafter(mids, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert O.e2m1_codes(np.array([-0.1, -0.0, -0.5, -5.1])).tolist() == [0, 0, 9, 15]
    assert O.e2m1_values(np.arange(16, dtype=np.uint8)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6,
                                                                    0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_quantise_scales_and_worst_rounding():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((500, 128)).astype(np.float32) * np.exp(rng.uniform(-6, 6, (500, 1))).astype(np.float32)
    code, s = O.quantise_f32(y)
    amax = np.abs(y).max(axis=1).astype(np.float64)
    assert np.all(np.abs(s.astype(np.float64) - amax / 6) <= amax / 6 * (2.0 ** -11 + 2.0 ** -24))
    back = O.e2m1_values(code) * s.astype(np.float64)[:, None]
    # levels lie at most 2 apart (4 to 6): off by at most one scale, and by what the scale lost at 6
    assert np.all(np.abs(back - y) <= s.astype(np.float64)[:, None] * (1 + 6 * 2.0 ** -10))
    code, s = O.quantise_f32(np.zeros((1, 64), np.float32))
    assert not code.any() and s[0] == 0


@pytest.mark.parametrize("style", [0, 1])
def test_angles_turn_pairs_and_keep_products(style):
    # the product of a query at p and a key at t depends on p - t alone
    rng = np.random.default_rng(1)
    half = 16
    ang = np.arange(64)[:, None] * (0.3 ** np.arange(half))
    table = np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)
    q, k = rng.standard_normal((2, 1, 1, 64)).astype(np.float32)

    def at(p, t):
        return float(np.sum(O.turn_f32(q, table[p:p + 1], style).astype(np.float64)
                            * O.turn_f32(k, table[t:t + 1], style)))
    assert abs(at(30, 10) - at(50, 30)) < 1e-4 and abs(at(30, 10) - at(31, 10)) > 1e-3
    assert np.array_equal(O.turn_f32(q, table[:1], style), q)                  # position 0: cos 1, sin 0


def test_rotation_is_the_hadamard_matrix():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 2, 256)).astype(np.float32)
    assert np.allclose(O.rotate_f32(x), O.rotate(x), rtol=0, atol=1e-4)
    H = O.hadamard()
    assert np.array_equal(H @ H.T, 128 * np.eye(128))


def test_norm_of_a_known_row():
    x = np.full((1, 128), 3.0, np.float32)
    h, n, mass = O.add_rmsnorm(x, x, np.ones(128, np.float32), 0.0, "f32", False)
    assert np.all(h == 6) and np.allclose(n, 1) and np.allclose(mass, 128)
    _, n, _ = O.add_rmsnorm(x, None, np.ones(128, np.float32), 0.0, "f32", True)
    assert np.allclose(n[0, 0], 128) and np.allclose(n[0, 1:], 0)


def test_cache_puts_and_gets_tokens():
    rng = np.random.default_rng(3)
    c = O.Cache(3, 2, 32, 64, rng)
    before = {t: c.get(1, t) for t in range(32) if t != 13}
    k, v = (O.quantise_f32(rng.standard_normal((2, 64)).astype(np.float32)) for _ in range(2))
    c.put(1, 13, k, v)
    got = c.get(1, 13)
    assert np.array_equal(got[0], O.e2m1_values(k[0]) * k[1].astype(np.float64)[:, None])
    assert np.array_equal(got[1], O.e2m1_values(v[0]) * v[1].astype(np.float64)[:, None])
    for t, (a, b) in before.items():
        assert np.array_equal(c.get(1, t)[0], a, equal_nan=True) and np.array_equal(c.get(1, t)[1], b, equal_nan=True)
    K, V, on = O.tokens_of(c, np.array([7, 1]), 46)
    assert not on[:32].any() and on[32:].all()
    assert np.array_equal(K[45], got[0]) and np.array_equal(V[45], got[1])


def test_attention_masks():
    rng = np.random.default_rng(4)
    c = O.Cache(4, 1, 32, 64)
    for p in range(4):
        for t in range(32):
            c.put(p, t, O.quantise_f32(rng.standard_normal((1, 64)).astype(np.float32)),
                  O.quantise_f32(rng.standard_normal((1, 64)).astype(np.float32)))
    table = np.array([[2, 0, -1]])
    q = rng.standard_normal((3, 2, 64)).astype(np.float32)
    out, _, _ = O.attention(q, c, table, np.array([40]), np.array([0, 3]), 0.1, True, 1)
    V = O.tokens_of(c, table[0], 40)[1]
    assert np.allclose(out[:, 0], V[37:40, 0]) and np.allclose(out[:, 1], V[37:40, 0])   # one token each: its value
    out, _, _ = O.attention(q, c, table, np.array([90]), np.array([0, 3]), 0.1, True, 20)
    assert np.all(out == 0)                                                    # tokens 64 .. are on an absent page
    out, _, _ = O.attention(q, c, table, np.array([2]), np.array([0, 3]), 0.1, True, 0)
    assert np.all(out[0] == 0) and np.all(np.isfinite(out))                    # the first row stands before token 0
