"""How well linear attention holds a term of its state, in the oracle's arithmetic: the bound that the GPU's states are held to
tells parts enough from too few."""
import numpy as np

from oracle import layer as O

# A state entry of one term, k_j v_j a^m, of rows with |g| <= 0.01 and at most 13 rows: the exponent's two roundings (2^-24 of less
# than 0.2 each) and exp2's (2^-23) at most three times, a product with each of them (2^-24), and two f16 parts' 2^-22.
STATE_TERM = 3 * (2 * 0.2 * 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -24) + 2.0 ** -22


def off(v, parts, round_to):
    """Largest error of v taken as a sum of `parts` rounded ones, relative to v."""
    rest = v.copy()
    for _ in range(parts):
        rest = rest - round_to(rest.astype(np.float32)).astype(np.float64)
    return np.max(np.abs(rest) / np.abs(v))


def test_parts_that_hold_an_aged_value():
    rng = np.random.default_rng(0)
    v = O.to_dtype(rng.standard_normal(4096), "f16").astype(np.float64) * np.exp(-0.01 * rng.integers(1, 12, 4096))
    v = (v * 2.0 ** np.round(14 - np.log2(np.abs(v)))).astype(np.float32).astype(np.float64)

    def f16(x):
        return x.astype(np.float16).astype(np.float32)
    assert off(v, 2, O.bf16_round) > 2 * STATE_TERM and off(v, 1, f16) > 2 * STATE_TERM
    assert off(v, 3, O.bf16_round) <= 2.0 ** -24 and off(v, 2, f16) <= 2.0 ** -22
