"""GPU: the token mixers at sizes that choose other launches than small calls do: many pairs of rows and heads over many steps,
selections of several lists a workgroup's share, sequences past one look of a wave; and rows that are no token, whose queries
may hold anything."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from oracle import mixers as X
from rotated_w8a8_int8_amd import binding as B
from test_gpu_attn_tree import check
from test_gpu_kv4_evict import run_select
from test_gpu_linear_attn import run as run_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def scaled_cache(rng, pages, heads, page, D):
    """Any codes, scales of keys about 0.3 and of values about 0.5."""
    c = O.Cache(pages, heads, page, D, rng)
    c.k_scale[:] = (0.3 * np.exp(rng.uniform(-0.5, 0.5, c.k_scale.shape))).astype(np.float16)
    c.v_scale[:] = (0.5 * np.exp(rng.uniform(-1, 1, c.v_scale.shape))).astype(np.float16)
    return c


def run_weights(torch, new, ctx, heads, G, D, page, dtype, causal=True, window=0, observe=0, factor=1.0, seed=0, pad=0, garbage=None,
                max_q=None):
    """As test_gpu_attn_tree.run_weights; garbage: what the queries of rows that are no token, past max_q or padding hold."""
    rng = np.random.default_rng(seed)
    start, seq_len = C.ragged(new), np.array(new) + np.array(ctx)
    T = int(start[-1]) + pad
    table, pages = C.page_table(rng, np.maximum(seq_len, 0), page)
    ref = scaled_cache(rng, pages, heads, page, D)
    q = O.to_dtype(rng.standard_normal((T, heads * G, D)), dtype)
    batch = C.device_batch(torch, table, seq_len, start, T, max_q)
    taken = np.zeros(T, bool)
    for b, n in enumerate(new):
        i = np.arange(n)
        taken[start[b]:start[b + 1]] = (seq_len[b] - n + i >= 0) & (i < (max_q or n))
    if garbage is not None:
        q[~taken] = garbage
    cap, sm = table.shape[1] * page, D ** -0.5
    old = rng.random((len(new), heads, cap)).astype(np.float32)
    w, o = C.put(torch, old), torch.full((T, heads * G, D), 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    B.attn_kv4_weights(C.device_cache(torch, ref), batch, C.put(torch, q, dtype), w, sm, causal=causal, window=window, observe=observe,
                       factor=factor, o=o)
    clean = np.where(taken[:, None, None], q, 0)
    want, mass, reach, p = X.attend(clean, ref, table, seq_len, start, sm, lambda b, n, m, on: X.sees_position(n, m, on, causal, window))
    got = C.host(o)
    if max_q:
        for b, n in enumerate(new):                           # later rows: left as they were, and counted for nothing
            assert np.all(got[start[b] + min(n, max_q):start[b + 1]] == 33.0)
            got[start[b] + min(n, max_q):start[b + 1]] = want[start[b] + min(n, max_q):start[b + 1]]
            for h in range(heads * G):
                if n:
                    p[b, h][max_q:] = 0
    check(got, want, mass, reach, dtype, seq_len, start, T)
    new_w, slack = X.weights(old, p, reach, heads, G, seq_len, start, observe, factor)
    n = max(1, int(seq_len.max()))                            # as derived in test_gpu_attn_tree.run_weights
    rel = (2 * np.sqrt(n) + 64 + max(new) * G / 32 + 22) * 2.0 ** -24 + 2.0 ** -21
    off, tol = np.abs(w.cpu().numpy() - new_w), slack + rel * np.abs(new_w) + 1e-30
    assert np.all(off <= tol), "weights off by %g of the tolerance" % np.nanmax(off / tol)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("garbage", [np.nan, np.inf, 1e30])
@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("new,G", [([4, 1, 6], 3), ([40, 9, 20], 3)])
def test_queries_of_rows_that_are_no_token(torch, new, G, dtype, garbage, causal):
    # the first rows of the sequences lie before token 0, the last rows of the call are padding
    if dtype == "f16" and garbage == 1e30:
        garbage = 6e4
    run_weights(torch, new, [-2, 30, -5], 2, G, 64, 32, dtype, causal, 0, 0, 0.5, seed=len(new), pad=3, garbage=garbage)
    run_weights(torch, new, [-2, 30, 5], 2, G, 64, 32, dtype, causal, 0, 0, 0.5, seed=len(new), pad=1, garbage=garbage, max_q=3)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("causal,window,observe", [(True, 0, 0), (False, 700, 6)])
def test_weights_of_many_pairs_over_many_steps(torch, D, dtype, causal, window, observe):
    # a step a wave: 10 rows of 5 heads, 32 (sequence, head) pairs, 129 steps and more
    print("many", D, dtype, causal, flush=True)
    run_weights(torch, [10, 7, 10, 0], [4100, 2000, 33, 3500], 8, 7, D, 64, dtype, causal, window, observe, 0.5, seed=D, pad=2)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("sequences,heads", [(20, 2), (40, 2), (70, 2)])
def test_selections_of_many_lists(torch, sequences, heads, kind):
    # 40, 80 and 140 lists of up to 17000 tokens: four, two and one workgroup a list
    print("lists", sequences, kind, flush=True)
    rng = np.random.default_rng(sequences)
    for longest, budget in ((5000, 700), (17000, 4000), (45000, 4001)):
        run_select(torch, rng.integers(longest // 3, longest, sequences).tolist() + [longest], heads, budget, 4, budget // 5, kind, seed=longest)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("sequences", [64, 65, 130, 700])
def test_linear_attention_of_many_ragged_sequences(torch, sequences, dtype):
    # a place's sequence is looked for 64 at a time
    rng = np.random.default_rng(sequences)
    new = rng.integers(0, 30, sequences)
    new[rng.choice(sequences, 3, replace=False)] = (200, 129, 400)
    run_linear(torch, new.tolist(), 2, 1, 64, dtype, seed=sequences, pad=1)
    run_linear(torch, new.tolist(), 40 if sequences < 200 else 4, 4, 64, dtype, seed=sequences, pad=1, in_place=True)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("rows", [3, 40])
def test_weights_of_more_sequences_than_are_looked_at_by_all(torch, rows, dtype):
    # past 512 sequences no context is cut, and tiles are found another way
    rng = np.random.default_rng(rows)
    new = rng.integers(0, rows, 600)
    run_weights(torch, new.tolist(), rng.integers(-3, 70, 600).tolist(), 1, 2, 64, 32, dtype, True, 0, 0, 0.5, seed=rows, pad=2)
