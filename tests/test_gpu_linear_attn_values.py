"""GPU: rad_linear_attn with values that are not finite, products that leave f32's range, and value columns, rows and states of
very different sizes: nothing reaches an earlier row, another sequence, or a head or column that it has no part in."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from oracle import mixers as X
from rotated_w8a8_int8_amd import binding as B
from test_gpu_linear_attn import tolerance
from test_oracle_linear_parts import STATE_TERM

pytestmark = pytest.mark.gpu
NEW = [70, 9, 40, 33]                                        # rows a sequence, in chunks and segments


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def inputs(seed, D, dtype, new, heads=4, qk=2):
    rng = np.random.default_rng(seed)
    T = sum(new)
    q, k, v = (O.to_dtype(rng.standard_normal((T, n, D)), dtype) for n in (qk, qk, heads))
    g = -np.exp2(rng.uniform(-8, -2, heads)).astype(np.float32)
    S = rng.standard_normal((len(new), heads, D, D)).astype(np.float32)
    return q, k, v, g, S


def call(torch, q, k, v, g, S, dtype, new, scale):
    o = torch.full(v.shape, 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    state = torch.full(S.shape, 44.0, device="cuda")
    B.linear_attn(C.put(torch, q, dtype), C.put(torch, k, dtype), C.put(torch, v, dtype), C.put(torch, g), state=C.put(torch, S),
                  state_out=state, q_start=C.put(torch, C.ragged(new)), max_q=max(new), scale=scale, o=o)
    return C.host(o), state.cpu().numpy()


def check(got, want, mass, S, want_S, big, dtype, new, D, rows=Ellipsis, states=Ellipsis):
    """Outputs at `rows` (of rows, heads, columns) and states at `states` (of sequences, heads, key dims, columns)."""
    to, ts = tolerance(dtype, max(new), D, 1.0, want, mass, want_S, big)
    off = np.abs(got - want)[rows]
    assert np.all(off <= to[rows]), "off by %g of the tolerance" % np.nanmax(off / to[rows])
    off = np.abs(S - want_S)[states]
    assert np.all(off <= ts[states]), "state off by %g of the tolerance" % np.nanmax(off / ts[states])


@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_what_is_not_finite_reaches_no_earlier_row_and_no_other_column(torch, what, bad, D, dtype):
    print("not finite", what, bad, D, dtype, flush=True)
    q, k, v, g, S = inputs(D, D, dtype, NEW)
    start, scale = C.ragged(NEW), D ** -0.5
    want, want_S, mass, big = X.linear(q, k, v, g, S, start, scale)
    # a row of the middle of the first sequence, of its first rows, and the last of the third one
    for seq, at in ((0, 45), (0, 5), (2, 39)):
        x = {"q": q.copy(), "k": k.copy(), "v": v.copy()}
        row, column = int(start[seq]) + at, D - 5
        x[what][row, 1, column] = bad
        got, state = call(torch, x["q"], x["k"], x["v"], g, S, dtype, NEW, scale)
        # what it has no part in: other rows (q), heads (k: of the other key head), columns (v), and all that came before
        clean, clean_S = np.ones(want.shape, bool), np.ones(S.shape, bool)
        after = slice(row, int(start[seq + 1]))
        if what == "q":
            clean[row, 2:] = False
        elif what == "k":
            clean[after, 2:], clean_S[seq, 2:] = False, False
        else:
            clean[after, 1, column], clean_S[seq, 1, :, column] = False, False
        check(got, want, mass, state, want_S, big, dtype, NEW, D, clean, clean_S)
        assert not np.isfinite(got[row, 1 if what == "v" else 2, column]), "the row itself"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
def test_products_with_later_rows_may_leave_the_range(torch, D, dtype):
    # finite inputs and finite exact outputs: only a query's product with a later row's key is past 2^128
    q, k, v, g, S = inputs(D + 1, D, dtype, NEW)
    start = C.ragged(NEW)
    for seq, early, late in ((0, 40, 60), (2, 2, 30)):         # rows of one chunk of 32
        q[start[seq] + early] *= np.float32(2.0 ** 80)
        k[start[seq] + late] *= np.float32(2.0 ** 60)
    want, want_S, mass, big = X.linear(q, k, v, g, S, start, 1.0)
    got, state = call(torch, q, k, v, g, S, dtype, NEW, 1.0)
    assert np.all(np.abs(want) < 2.0 ** 126)
    check(got, want, mass, state, want_S, big, dtype, NEW, D)


def columns_of_size(D, lo, hi):
    """A power of two a value column, from 2^lo to 2^hi, neighbours far apart."""
    return np.exp2(np.round(np.linspace(lo, hi, D))[np.arange(D) * 37 % D]).astype(np.float32)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
def test_value_columns_of_very_different_sizes(torch, D, dtype):
    # each column, and its part of the state, is as good as if it were alone
    q, k, v, g, S = inputs(D + 2, D, dtype, NEW)
    size = columns_of_size(D, -13, 13)
    v, S = O.to_dtype(v * size, dtype), S * size
    scale = 2.0 ** -5
    want, want_S, mass, big = X.linear(q, k, v, g, S, C.ragged(NEW), scale)
    got, state = call(torch, q, k, v, g, S, dtype, NEW, scale)
    keep = np.abs(want) < 6e4                                 # f16 ends there
    check(got, want, mass, state, want_S, big, dtype, NEW, D, keep)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
def test_query_rows_of_very_different_sizes(torch, D, dtype):
    q, k, v, g, S = inputs(D + 3, D, dtype, NEW)
    size = np.exp2(np.round(np.linspace(-13, 13, len(q)))[np.arange(len(q)) * 37 % len(q)])[:, None, None]
    q = O.to_dtype(q * size, dtype)
    want, want_S, mass, big = X.linear(q, k, v, g, S, C.ragged(NEW), 2.0 ** -5)
    got, state = call(torch, q, k, v, g, S, dtype, NEW, 2.0 ** -5)
    check(got, want, mass, state, want_S, big, dtype, NEW, D, np.abs(want) < 6e4)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("size", [2.0 ** 64, 2.0 ** 110, 2.0 ** -64, 2.0 ** -110])
def test_states_far_from_the_values(torch, size, dtype):
    # values of 2^-20 meet states of 2^110; outputs come to about 1
    q, k, v, g, S = inputs(4, 64, dtype, NEW)
    q[5], q[45] = 0.0, 0.0
    v, S, scale = O.to_dtype(v * np.float32(2.0 ** -20), dtype), S * np.float32(size), min(1 / size, 1.0)
    want, want_S, mass, big = X.linear(q, k, v, g, S, C.ragged(NEW), scale)
    got, state = call(torch, q, k, v, g, S, dtype, NEW, scale)
    check(got, want, mass, state, want_S, big, dtype, NEW, 64)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
def test_many_values_that_are_not_finite(torch, D, dtype):
    # in several columns, rows and chunks, each from its own row on; zero keys and weights too, and rows behind a whole chunk
    q, k, v, g, S = inputs(D + 4, D, dtype, [150, 33])
    rng, start, scale = np.random.default_rng(D), C.ragged([150, 33]), D ** -0.5
    want, want_S, mass, big = X.linear(q, k, v, g, S, start, scale)
    clean, clean_S = np.ones(want.shape, bool), np.ones(S.shape, bool)
    for seq, lo, hi in ((0, 0, 150), (1, 150, 183)):
        for column in rng.choice(D, D // 3, replace=False):
            head, row = int(rng.integers(4)), int(rng.integers(lo, hi))
            v[row, head, column] = rng.choice([np.nan, np.inf, -np.inf])
            clean[row:hi, head, column], clean_S[seq, head, :, column] = False, False
    got, state = call(torch, q, k, v, g, S, dtype, [150, 33], scale)
    check(got, want, mass, state, want_S, big, dtype, [150, 33], D, clean, clean_S)
    assert not np.isfinite(got[~clean]).any() and not np.isfinite(state[~clean_S]).any()


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
def test_states_hold_more_than_the_values_type(torch, D, dtype):
    # rows whose keys are 0 but one row's: nothing is added up, so that each entry shows how well a term is held
    rng, n, heads = np.random.default_rng(D), 13, 4
    q, k, v = (O.to_dtype(rng.standard_normal((n, x, D)), dtype) for x in (2, 2, heads))
    j = int(rng.integers(n))
    k[np.arange(n) != j] = 0
    g = -rng.uniform(0.002, 0.01, heads).astype(np.float32)
    _, state = call(torch, q, k, v, g, np.zeros((1, heads, D, D), np.float32), dtype, [n], 1.0)
    want = X.linear(q, k, v, g, np.zeros((1, heads, D, D)), np.array([0, n]), 1.0)[1]
    assert np.all(np.abs(state - want) <= STATE_TERM * np.abs(want) + 1e-30), np.max(np.abs(state - want) / np.maximum(np.abs(want), 1e-30))


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_what_is_not_finite_row_by_row(torch, what, D, dtype):
    new = [3, 1, 0, 8]
    q, k, v, g, S = inputs(D + 5, D, dtype, new)
    start, scale = C.ragged(new), D ** -0.5
    want, want_S, mass, big = X.linear(q, k, v, g, S, start, scale)
    x = {"q": q, "k": k, "v": v}
    x[what][6, 1, 7] = np.nan
    got, state = call(torch, x["q"], x["k"], x["v"], g, S, dtype, new, scale)
    clean, clean_S = np.ones(want.shape, bool), np.ones(S.shape, bool)
    if what == "q":
        clean[6, 2:] = False
    elif what == "k":
        clean[6:, 2:], clean_S[3, 2:] = False, False
    else:
        clean[6:, 1, 7], clean_S[3, 1, :, 7] = False, False
    check(got, want, mass, state, want_S, big, dtype, new, D, clean, clean_S)
    assert not np.isfinite(got[~clean]).any()
