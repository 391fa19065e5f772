"""GPU: rad_attn_kv4_tree against attention in 64 bits under the same masks, every element within the derived tolerance of
the causal form's tests; and rad_attn_kv4_weights: outputs alike, weights within a bound derived here."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from oracle import mixers as X
from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def tree_masks(rng, n, words, kind):
    """uint64 [n][words]: a random tree's ancestors ("tree"), any bits at all ("any"), none ("none"), a block ("all")."""
    m = np.zeros((n, words), np.uint64)
    if kind == "any":
        return rng.integers(0, 1 << 63, (n, words)).astype(np.uint64) * np.uint64(2) + rng.integers(0, 2, (n, words)).astype(np.uint64)
    if kind == "all":
        return ~m
    if kind == "tree":
        for i in range(n):
            parent = int(rng.integers(max(-1, i - 5), i)) if i else -1
            if parent >= 0:
                m[i] = m[parent]
            if i < 64 * words:
                m[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return m


def setup(torch, new, ctx, heads, G, D, page, dtype, seed, pad=0, edit=None, max_q=None, q_size=2.0, width=None):
    rng = np.random.default_rng(seed)
    start = C.ragged(new)
    T = int(start[-1]) + pad
    seq_len = np.array(new) + np.array(ctx)
    table, pages = C.page_table(rng, np.maximum(seq_len, 0), page, width)
    if edit is not None:
        edit(table, pages)
    ref = O.Cache(pages, heads, page, D, rng)
    C.fill_cache(rng, ref, table, np.maximum(seq_len, 0))
    q = O.to_dtype(q_size * rng.standard_normal((T, heads * G, D)), dtype)
    batch = C.device_batch(torch, table, seq_len, start, T, max_q)
    return rng, start, T, seq_len, table, ref, q, batch


def check(got, want, mass, reach, dtype, seq_len, start, T):
    padding = np.isnan(want)
    assert np.array_equal(padding[:, 0, 0], np.arange(T) >= start[-1])
    assert np.all(got[padding] == 33.0), "padding rows were written"
    tol = C.attention_tolerance(dtype, np.nan_to_num(want), mass, reach, max(1, int(seq_len.max())))
    off = np.where(padding, 0, np.abs(got - want))
    assert np.all(off <= tol), "off by %g of the tolerance at %s" % (np.max(off / tol), np.unravel_index(np.argmax(off / tol), off.shape))


def run_tree(torch, new, ctx, heads, G, D, page, dtype, kind="tree", words=None, window=0, seed=0, pad=0, edit=None):
    rng, start, T, seq_len, table, ref, q, batch = setup(torch, new, ctx, heads, G, D, page, dtype, seed, pad, edit)
    words = (max(new) + 63) // 64 if words is None else words
    mask = np.concatenate([tree_masks(rng, n, words, kind) for n in new] + [tree_masks(rng, pad, words, "any")])
    o = torch.full((T, heads * G, D), 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    sm = D ** -0.5
    B.attn_kv4_tree(C.device_cache(torch, ref), batch, C.put(torch, q, dtype), C.put(torch, mask.view(np.int64)), sm, window=window, o=o)
    want, mass, reach, _ = X.attend(q, ref, table, seq_len, start, sm,
                                    lambda b, n, m, on: X.sees_tree(n, m, on, mask[start[b]:start[b] + n], window))
    check(C.host(o), want, mass, reach, dtype, seq_len, start, T)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("kind", ["tree", "any", "none", "all"])
@pytest.mark.parametrize("D,G,page", [(64, 8, 32), (128, 5, 64), (256, 3, 128), (128, 1, 256)])
def test_ragged_trees(torch, D, G, page, kind, dtype):
    print("tree", D, G, page, kind, dtype, flush=True)
    run_tree(torch, [16, 3, 0, 7, 1, 12], [100, 0, 50, 61, 33, -5], 2, G, D, page, dtype, kind, seed=D + G, pad=3)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("n,ctx", [(1, 0), (1, 31), (3, 1000), (32, 32), (33, 0), (64, 300), (65, 7), (130, 90)])
def test_every_size_near_a_word_and_a_step(torch, n, ctx, dtype):
    print("size", n, ctx, dtype, flush=True)
    run_tree(torch, [n], [ctx], 2, 4, 128, 64, dtype, "tree", seed=n)
    run_tree(torch, [n], [ctx], 1, 2, 64, 32, dtype, "any", words=(n + 63) // 64 + 1, seed=n + 1)


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("window", [1, 7, 40, 100000])
def test_windows(torch, window, kind):
    run_tree(torch, [9, 20, 4], [70, 10, 0], 2, 3, 64, 32, "f32", kind, window=window, seed=window)
    run_tree(torch, [60], [300], 1, 5, 128, 64, "bf16", kind, window=window, seed=window + 1)


def test_nodes_past_the_words_are_not_seen(torch):
    run_tree(torch, [100, 70], [40, 3], 2, 2, 64, 32, "f32", "all", words=1, seed=5)


def test_absent_pages(torch):
    def edit(table, pages):
        table[0, 1], table[0, 3], table[1, 0] = -1, pages + 5, 1 << 30
    run_tree(torch, [8, 12], [120, 60], 2, 4, 128, 32, "bf16", "tree", seed=8, edit=edit)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_sequences(torch, dtype):
    # past 512 sequences tiles are found another way
    rng = np.random.default_rng(3)
    new = rng.integers(0, 9, 600).tolist()
    run_tree(torch, new, rng.integers(0, 40, 600).tolist(), 1, 3, 64, 32, dtype, "tree", seed=3, pad=2)


def test_a_chain_gives_what_causal_attention_gives(torch):
    for n, ctx, window in ((5, 2000, 0), (40, 300, 64)):
        rng, start, T, seq_len, table, ref, q, batch = setup(torch, [n, 3], [ctx, 9], 2, 4, 128, 64, "bf16", seed=n)
        mask = np.concatenate([[(1 << (i + 1)) - 1 for i in range(k)] for k in (n, 3)]).astype(np.uint64)[:, None]
        cache, qd = C.device_cache(torch, ref), C.put(torch, q, "bf16")
        a = B.attn_kv4(cache, batch, qd, 0.09, window=window)
        b = B.attn_kv4_tree(cache, batch, qd, C.put(torch, mask.view(np.int64)), 0.09, window=window)
        # the same products in the same order wherever the cut is the same; else within a rounding of the output
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=2.0 ** -7 * float(a.float().abs().max()))


# --------------------------------------------------------------------------------------------- weights --

def run_weights(torch, new, ctx, heads, G, D, page, dtype, causal=True, window=0, observe=0, factor=1.0, seed=0, pad=0,
                edit=None, one=False, extra=0, times=1):
    rng, start, T, seq_len, table, ref, q, batch = setup(torch, new, ctx, heads, G, D, page, dtype, seed, pad, edit)
    if one:
        batch = C.device_batch(torch, table, seq_len, None, T)
    cap = table.shape[1] * page
    old = rng.random((len(new), heads, cap + extra)).astype(np.float32)
    if factor == 0:
        old[:] = np.nan
    else:
        # what the call's own tokens find is not read either
        for b, n in enumerate(new):
            old[b, :, max(int(seq_len[b]) - n, 0):int(max(seq_len[b], 0))] = np.nan
    w, sm = C.put(torch, old), D ** -0.5
    o = torch.full((T, heads * G, D), 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    cache, qd = C.device_cache(torch, ref), C.put(torch, q, dtype)
    B.attn_kv4_weights(cache, batch, qd, w, sm, causal=causal, window=window, observe=observe, factor=factor, o=o)
    want, mass, reach, p = X.attend(q, ref, table, seq_len, start, sm, lambda b, n, m, on: X.sees_position(n, m, on, causal, window))
    check(C.host(o), want, mass, reach, dtype, seq_len, start, T)
    new_w, slack = X.weights(old, p, reach, heads, G, seq_len, start, observe, factor)
    got = w.cpu().numpy()
    kept = np.isnan(new_w)
    assert np.array_equal(np.isnan(got), kept)
    for b, n in enumerate(new):
        if n == 0:
            assert np.array_equal(got[b], old[b], equal_nan=True), "a sequence without rows"
        L = int(np.clip(seq_len[b], 0, cap))
        assert np.array_equal(got[b, :, L:], old[b, :, L:], equal_nan=True), "past the length"
    # A probability is off by a factor of at most expm1(2 e), e = 2^-14 reach (a score and the normaliser: slack), by the
    # f32 sum of the normaliser (2 sqrt(n) + 64 roundings, as in layer_cases.attention_tolerance) and by exp2 and two
    # products (2^-21).  A wave sums 16 of a tile of 32 pairs in a lane, then the tiles, then two lanes: pairs / 32 + 20
    # roundings at most; the fading product and sum two more.
    n = max(1, int(seq_len.max()))
    rel = (2 * np.sqrt(n) + 64 + max(new) * G / 32 + 22) * 2.0 ** -24 + 2.0 ** -21
    tol = slack + rel * np.abs(new_w) + 1e-30
    off = np.where(kept, 0, np.abs(got - new_w))
    assert np.all(off <= np.where(kept, 1, tol)), "weights off by %g of the tolerance" % np.nanmax(off / tol)
    again = C.put(torch, old)
    B.attn_kv4_weights(cache, batch, qd, again, sm, causal=causal, window=window, observe=observe, factor=factor, o=o)
    assert np.array_equal(again.cpu().numpy(), got, equal_nan=True), "another run, another sum"


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D,G,page", [(64, 8, 32), (128, 5, 64), (256, 3, 128), (128, 40, 64)])
def test_weights_of_single_tokens(torch, D, G, page, dtype):
    print("weights", D, G, page, dtype, flush=True)
    run_weights(torch, [1, 1, 1, 1, 1], [0, 1, 31, 77, 300], 2, G, D, page, dtype, seed=D + G, one=True, extra=8)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("causal,window,observe,factor", [(True, 0, 0, 1.0), (True, 0, 3, 0.0), (False, 0, 0, 0.5),
                                                         (True, 20, 0, 0.9), (True, 9, 5, 1.0), (False, 30, 2, 0.25)])
def test_weights_of_blocks_and_prompts(torch, causal, window, observe, factor, dtype):
    print("weights", causal, window, observe, factor, dtype, flush=True)
    run_weights(torch, [16, 3, 0, 7, 1, 12], [100, 0, 50, 61, 33, -5], 2, 3, 64, 32, dtype, causal, window, observe, factor,
                seed=int(10 * factor), pad=3)
    run_weights(torch, [150, 40], [10, 200], 1, 5, 128, 64, dtype, causal, window, observe, factor, seed=int(10 * factor) + 1)


def test_weights_of_a_long_context(torch):
    run_weights(torch, [1], [9000], 1, 4, 64, 64, "f32", seed=1, one=True)
    run_weights(torch, [4, 2], [6000, 2500], 1, 2, 64, 32, "bf16", factor=0.5, seed=2)


@pytest.mark.parametrize("sequences", [2, 63, 64, 65])
def test_weights_of_sequences_of_very_different_lengths(torch, sequences):
    # up to 64 sequences share the workgroups by their lengths
    ctx = [3000] + [(37 * i) % 150 for i in range(sequences - 2)] + [700]
    new = [1] + [i % 3 for i in range(sequences - 2)] + [2]
    run_weights(torch, new, ctx, 2, 2, 64, 32, "f16", factor=0.5, seed=sequences, pad=1)
    run_weights(torch, [1] * sequences, ctx, 1, 20, 64, 64, "bf16", seed=sequences, one=True)


def test_weights_on_absent_pages(torch):
    def edit(table, pages):
        table[0, 1], table[1, 0] = -1, pages + 3
    run_weights(torch, [4, 3], [120, 60], 2, 4, 128, 32, "f32", seed=8, edit=edit, factor=0.5)


def test_far_scores_stay_finite(torch):
    # scores past 2^22, where f32 holds the reference exponent to half a unit or worse
    rng, start, T, seq_len, table, ref, q, batch = setup(torch, [3], [200], 1, 4, 64, 32, "f32", 4, q_size=3e6)
    w = torch.zeros((1, 1, table.shape[1] * 32), device="cuda")
    o, _ = B.attn_kv4_weights(C.device_cache(torch, ref), batch, C.put(torch, q), w, 1.0, factor=0.0)
    assert torch.isfinite(o).all() and torch.isfinite(w).all()
    assert abs(float(w.sum()) - 12) < 12 * 2.0 ** -10          # 3 rows of 4 heads
