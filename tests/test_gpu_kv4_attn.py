"""GPU: rad_attn_kv4 against attention in 64 bits over the same cache, every element within a derived tolerance:
types, head sizes and groupings, lengths from none to many pages, ragged batches, masks, absent pages, stale memory."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def run(torch, new, ctx, heads, G, D, page, dtype, causal=True, window=0, seed=0, pad=0, table_edit=None, width=None,
        q_size=2.0, k_size=1.0, max_q=None, plain=False):
    rng = np.random.default_rng(seed)
    start = C.ragged(new)
    T = int(start[-1]) + pad
    seq_len = np.array(new) + np.array(ctx)
    table, pages = C.page_table(rng, np.maximum(seq_len, 0), page, width)
    if table_edit is not None:
        table_edit(table, pages)
    ref = O.Cache(pages, heads, page, D, rng)
    C.fill_cache(rng, ref, table, np.maximum(seq_len, 0), k_size)
    q = O.to_dtype(q_size * rng.standard_normal((T, heads * G, D)), dtype)
    one = all(n == 1 for n in new) and pad == 0 and not plain
    batch = C.device_batch(torch, table, seq_len, None if one else start, T, max_q)
    sm = D ** -0.5
    o = torch.full((T, heads * G, D), 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    B.attn_kv4(C.device_cache(torch, ref), batch, C.put(torch, q, dtype), sm, causal=causal, window=window, o=o)
    got = C.host(o)
    want, mass, reach = O.attention(q, ref, table, seq_len, start, sm, causal, window)
    padding = np.isnan(want)
    assert np.array_equal(padding[:, 0, 0], np.arange(T) >= start[-1])
    assert np.all(got[padding] == 33.0), "padding rows were written"
    tol = C.attention_tolerance(dtype, np.nan_to_num(want), mass, reach, max(1, int(seq_len.max())))
    off = np.abs(got - want)
    off[padding] = 0
    assert np.all(off <= tol), "off by %g of the tolerance at %s" % (np.max(off / tol), np.unravel_index(np.argmax(off / tol), off.shape))


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("G", [1, 4, 5, 8, 11, 16, 20])
def test_one_token_a_sequence(torch, G, D, dtype):
    print("decode", G, D, dtype, flush=True)
    run(torch, [1, 1, 1, 1, 1], [0, 1, 31, 77, 300], 2, G, D, 32, dtype, seed=G + D)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 1000])
def test_every_length_near_a_tile(torch, n, dtype):
    print("length", n, dtype, flush=True)
    run(torch, [1], [n - 1], 1, 5, 128, 64, dtype, seed=n)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,G,page", [(64, 8, 32), (128, 5, 64), (256, 3, 128), (128, 1, 256)])
def test_ragged_blocks(torch, D, G, page, causal, dtype):
    print("blocks", D, G, page, causal, dtype, flush=True)
    run(torch, [16, 3, 0, 7, 1], [100, 0, 50, 61, 33], 2, G, D, page, dtype, causal, seed=D + G, pad=3)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("n,ctx", [(97, 0), (130, 5), (200, 128), (257, 40)])
def test_prompts(torch, n, ctx, dtype):
    print("prompt", n, ctx, dtype, flush=True)
    run(torch, [n, 1], [ctx, 90], 2, 5, 128, 64, dtype, seed=n)
    run(torch, [n], [ctx], 1, 2, 64, 32, dtype, causal=False, seed=n + 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 7, 32, 100, 5000])
def test_windows(torch, window, dtype):
    print("window", window, dtype, flush=True)
    run(torch, [1, 1], [200, 3], 2, 4, 128, 32, dtype, window=window, seed=window)
    run(torch, [40, 9], [150, 0], 1, 5, 64, 32, dtype, window=window, seed=window + 1)
    run(torch, [20, 9], [150, 0], 1, 5, 128, 64, dtype, causal=False, window=window, seed=window + 2)
    run(torch, [160], [90], 1, 3, 128, 64, dtype, window=window, seed=window + 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_absent_pages_and_empty_rows(torch, dtype):
    def edit(table, pages):
        table[0, 0] = -1                                       # the first tokens are gone
        table[1, :] = pages + 5                                # all of them are
        table[2, 1] = -7
    run(torch, [1, 1, 1], [100, 60, 90], 2, 5, 128, 32, dtype, table_edit=edit)
    run(torch, [20, 4, 30], [100, 60, 70], 2, 5, 128, 32, dtype, table_edit=edit)
    run(torch, [20, 4, 30], [20, 60, 70], 2, 5, 64, 32, dtype, causal=False, table_edit=edit)
    run(torch, [6, 40], [-3, -25], 2, 5, 128, 32, dtype)       # rows before the first token: zeros
    run(torch, [1, 1], [-1, 10], 2, 5, 128, 32, dtype)         # an empty sequence


def test_lengths_past_the_table_are_cut(torch):
    rng = np.random.default_rng(1)
    ref = O.Cache(3, 1, 32, 128, rng)
    table = np.array([[0, 2]], np.int32)
    C.fill_cache(rng, ref, table, [64])
    q = rng.standard_normal((1, 4, 128)).astype(np.float32)
    dev = C.device_cache(torch, ref)
    a = B.attn_kv4(dev, C.device_batch(torch, table, [64], None, 1), C.put(torch, q), 0.1)
    b = B.attn_kv4(dev, C.device_batch(torch, table, [2 ** 31 - 1], None, 1), C.put(torch, q), 0.1)
    assert torch.equal(a, b)
    z = B.attn_kv4(dev, C.device_batch(torch, table, [-5], None, 1), C.put(torch, q), 0.1)
    assert not z.any()


@pytest.mark.parametrize("dtype", C.DTYPES)
def test_peaked_and_flat_scores(torch, dtype):
    # one token takes all, or all are alike; scores far beyond exp's range
    run(torch, [1, 1], [500, 90], 1, 5, 128, 64, dtype, q_size=30.0, k_size=4.0, seed=3)
    run(torch, [1, 1], [500, 90], 1, 5, 128, 64, dtype, q_size=0.0, seed=4)
    run(torch, [130], [70], 1, 5, 128, 64, dtype, q_size=30.0, k_size=4.0, seed=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_that_rise_with_the_context(torch, dtype):
    # every tile brings a new maximum: the running sums are rescaled each time
    rng = np.random.default_rng(7)
    n, D, page = 700, 128, 64
    ref = O.Cache(11, 1, page, D, rng)
    table = rng.permutation(11).astype(np.int32)[None]
    for t in range(n):
        k = np.full((1, D), 0.02 * t) + 0.1 * rng.standard_normal((1, D))
        v = rng.standard_normal((1, D)) * np.exp(rng.uniform(-6, 6))
        ref.put(int(table[0, t // page]), t % page, O.quantise_f32(k.astype(np.float32)),
                O.quantise_f32(v.astype(np.float32)))
    for rows in (1, 30):
        q = O.to_dtype(np.full((rows, 5, D), 1.0) + 0.1 * rng.standard_normal((rows, 5, D)), dtype)
        start = C.ragged([rows])
        got = C.host(B.attn_kv4(C.device_cache(torch, ref), C.device_batch(torch, table, [n], start, rows),
                                C.put(torch, q, dtype), 0.5))
        want, mass, reach = O.attention(q, ref, table, np.array([n]), start, 0.5, True, 0)
        assert np.all(np.abs(got - want) <= C.attention_tolerance(dtype, want, mass, reach, n))


def test_a_long_context(torch):
    # 70,001 tokens of one sequence: the context is split over workgroups and joined
    rng = np.random.default_rng(11)
    n, D, page, H, G = 70001, 128, 256, 1, 5
    pages = (n + page - 1) // page
    ref = O.Cache(pages, H, page, D, rng)
    ref.k_scale[:] = (0.2 * np.exp(rng.uniform(-0.3, 0.3, ref.k_scale.shape))).astype(np.float16)
    ref.v_scale[:] = (0.5 * np.exp(rng.uniform(-1, 1, ref.v_scale.shape))).astype(np.float16)
    table = rng.permutation(pages).astype(np.int32)[None]
    q = rng.standard_normal((1, G, D)).astype(np.float32)
    got = C.host(B.attn_kv4(C.device_cache(torch, ref), C.device_batch(torch, table, [n], None, 1), C.put(torch, q),
                            D ** -0.5))
    want, mass, reach = O.attention(q, ref, table, np.array([n]), C.ragged([1]), D ** -0.5, True, 0)
    assert np.all(np.abs(got - want) <= C.attention_tolerance("f32", want, mass, reach, n))


def test_rows_past_max_q_are_left(torch):
    rng = np.random.default_rng(2)
    ref = O.Cache(4, 1, 32, 64, rng)
    table = np.array([[0, 1]], np.int32)
    C.fill_cache(rng, ref, table, [50])
    q = C.put(torch, rng.standard_normal((10, 2, 64)).astype(np.float32))
    dev, o = C.device_cache(torch, ref), torch.full((10, 2, 64), 5.0, device="cuda")
    B.attn_kv4(dev, C.device_batch(torch, table, [50], C.ragged([10]), 10, max_q=4), q, 0.1, o=o)
    full = B.attn_kv4(dev, C.device_batch(torch, table, [50], C.ragged([10]), 10), q, 0.1)
    assert bool((o[4:] == 5).all())
    assert float((o[:4] - full[:4]).abs().max()) <= 1e-4


@pytest.mark.parametrize("n", [1, 40])
def test_extreme_factors_of_zero_scores(torch, n):
    # zero scores stay zero under the largest factor and beside a huge query element: every token weighs the same
    rng = np.random.default_rng(13)
    ref = O.Cache(2, 1, 32, 64)
    table = np.array([[0, 1]], np.int32)
    C.fill_cache(rng, ref, table, [50])
    ref.k_codes[..., 31] &= 0x0F                               # keys have no last dimension
    q = np.zeros((n, 2, 64), np.float32)
    q[:, 1, 63] = 1.0e38
    want, mass, reach = O.attention(np.zeros_like(q), ref, table, [50], C.ragged([n]), 1.0, False, 0)
    batch = C.device_batch(torch, table, [50], C.ragged([n]), n)
    for sm in (2.0 ** 126, 2.0 ** 20, 1e-38):
        got = C.host(B.attn_kv4(C.device_cache(torch, ref), batch, C.put(torch, q), sm, causal=False))
        assert np.all(np.abs(got - want) <= C.attention_tolerance("f32", want, mass, reach, 50)), sm


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("n", [1, 3, 40])
def test_rows_that_are_not_finite_keep_to_themselves(torch, n, dtype):
    # a row and head of NaN or infinite queries shares its products with others: theirs are as without it
    rng = np.random.default_rng(14)
    ref = O.Cache(6, 2, 32, 128)
    table = np.array([[4, 0, 2, 1, 5, 3]], np.int32)
    C.fill_cache(rng, ref, table, [170])
    q = O.to_dtype(rng.standard_normal((n, 8, 128)), dtype)
    batch, dev = C.device_batch(torch, table, [170], C.ragged([n]), n), C.device_cache(torch, ref)
    clean = C.host(B.attn_kv4(dev, batch, C.put(torch, q, dtype), 0.1))
    q[n // 2, 1, 7], q[0, 6, 100] = np.nan, np.inf
    got = C.host(B.attn_kv4(dev, batch, C.put(torch, q, dtype), 0.1))
    keep = np.ones((n, 8), bool)
    keep[n // 2, 1] = keep[0, 6] = False
    want, mass, reach = O.attention(np.where(np.isfinite(q), q, 0), ref, table, [170], C.ragged([n]), 0.1, True, 0)
    tol = C.attention_tolerance(dtype, want, mass, reach, 170)
    assert np.all(np.abs(got - want)[keep] <= tol[keep]) and np.all(np.abs(clean - want)[keep] <= tol[keep])


@pytest.mark.parametrize("n", [1, 24])
def test_pages_that_sequences_share(torch, n):
    # a common prefix, and one page twice in a row's table
    rng = np.random.default_rng(15)
    ref = O.Cache(5, 2, 32, 64)
    own = np.array([[0, 1, 2, 3, 4]], np.int32)
    C.fill_cache(rng, ref, own, [160])
    table = np.array([[0, 1, 2, -1], [0, 1, 3, 4], [2, 2, 2, 0]], np.int32)
    seq_len, start = np.array([90, 128, 100]), C.ragged([n] * 3)
    q = O.to_dtype(rng.standard_normal((3 * n, 4, 64)), "bf16")
    got = C.host(B.attn_kv4(C.device_cache(torch, ref), C.device_batch(torch, table, seq_len, start, 3 * n),
                            C.put(torch, q, "bf16"), 0.125))
    want, mass, reach = O.attention(q, ref, table, seq_len, start, 0.125, True, 0)
    assert np.all(np.abs(got - want) <= C.attention_tolerance("bf16", want, mass, reach, 128))


def test_nothing_to_attend_to(torch):
    dev = B.KV4Cache.empty(1, 2, 32, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    none = B.KVBatch(torch.zeros(0, 4, **i32), torch.zeros(0, **i32))
    q = torch.zeros(0, 4, 64, device="cuda")
    assert B.attn_kv4(dev, none, q, 0.1).shape == (0, 4, 64)
    k = torch.zeros(0, 2, 64, device="cuda")
    assert B.kv4_append(dev, none, k, k, q, rotate=False).shape == (0, 4, 64)
    assert B.kv4_read(dev, none)[0].shape == (0, 2, 64)
    # a table without pages: every row sees nothing
    bare = B.KVBatch(torch.zeros(2, 0, **i32), torch.full((2,), 9, **i32))
    assert not B.attn_kv4(dev, bare, torch.ones(2, 4, 64, device="cuda"), 0.1).any()


def test_the_same_call_twice_gives_the_same_bits(torch):
    rng = np.random.default_rng(12)
    ref = O.Cache(40, 2, 64, 128, rng)
    ref.k_scale[:], ref.v_scale[:] = np.float16(0.1), np.float16(0.3)
    table = rng.permutation(40).reshape(2, 20).astype(np.int32)
    dev = C.device_cache(torch, ref)
    for new in ([1, 1], [16, 5], [300, 200]):
        q = C.put(torch, rng.standard_normal((sum(new), 10, 128)).astype(np.float32))
        batch = C.device_batch(torch, table, [1200, 900], C.ragged(new), sum(new))
        assert torch.equal(B.attn_kv4(dev, batch, q, 0.1), B.attn_kv4(dev, batch, q, 0.1))


def test_binding_refusals(torch):
    dev = B.KV4Cache.empty(2, 2, 32, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = B.KVBatch(torch.zeros(1, 1, **i32), torch.ones(1, **i32))
    q = torch.zeros(1, 4, 64, device="cuda")
    with pytest.raises(ValueError, match="q has shape"):
        B.attn_kv4(dev, batch, torch.zeros(2, 4, 64, device="cuda"), 0.1)
    with pytest.raises(B.RadError):
        B.attn_kv4(dev, batch, torch.zeros(1, 3, 64, device="cuda"), 0.1)
    with pytest.raises(TypeError, match="o must be"):
        B.attn_kv4(dev, batch, q, 0.1, o=q.half())
    with pytest.raises(B.RadError):
        B.attn_kv4(dev, batch, q, 0.0)
    with pytest.raises(B.RadError):
        B.attn_kv4(dev, batch, q, 0.1, window=-3)


@pytest.mark.parametrize("gap", [14, 16, 18, 20, 22, 24])
@pytest.mark.parametrize("n,rows,D", [(200001, 1, 128), (200001, 12, 64), (200001, 40, 128), (1000, 1, 64), (1000, 12, 128),
                                      (1000, 12, 256), (1000, 40, 64), (1000, 40, 128)])
def test_a_peak_above_many_small_weights(torch, n, rows, D, gap):
    """f32: one token `gap` nats above all others, with a value in dimension 0 alone: what the others are worth
    together must not be lost with each of them.  The context is not cut (600 sequences, one of them long), so that a
    wave, whose weights share a scale, has a quarter of it.

    Of the mass of a dimension: the scores, 0 and `gap`, are right to 2^-21 (two f16 parts of the query, three
    roundings), the weights to 24 * 2^-21 for that and 2^-21 for their two parts; each of a wave's tokens adds one
    rounding to its sums, the join of the waves and the quotient at most 16, 2^-24 each.  Then a weight is off by up to
    2^-33 of the largest that it is held with, whatever the dimension's mass: of 6 for each of the tokens."""
    rng = np.random.default_rng(gap + D)
    page, others = 256, 599
    pages = (n + page - 1) // page
    ref = O.Cache(pages, 1, page, D)
    ref.k_scale[:], ref.v_scale[:] = 1, 1
    ref.v_codes[:] = 0xFF                                      # level 6, negative, in every dimension
    table = rng.permutation(pages).astype(np.int32)[None].repeat(others + 1, axis=0)
    at = int(rng.integers(0, 32))                              # the peak comes first: all that follows meets its scale
    key, value = np.zeros((1, D), np.uint8), np.zeros((1, D), np.uint8)
    key[0, 0] = value[0, 0] = 7
    ref.put(int(table[0, at // page]), at % page, (key, np.float16([1])), (value, np.float16([1])))
    q = np.zeros((rows + others, 1, D), np.float32)
    q[:, 0, 0] = gap / 6
    start, seq_len = C.ragged([1] * others + [rows]), np.array([0] * others + [n])
    got = C.host(B.attn_kv4(C.device_cache(torch, ref), C.device_batch(torch, table, seq_len, start, rows + others, rows),
                            C.put(torch, q), 1.0, causal=False))
    assert not got[:others].any()
    top, rest = np.exp(float(np.float32(gap / 6)) * 6), n - 1.0
    want, mass = np.full(D, -6 * rest / (top + rest)), np.full(D, 6 * rest / (top + rest))
    want[0], mass[0] = 6 * (top - rest) / (top + rest), 6
    tol = mass * (25 * 2.0 ** -21 + (n / 4 + 16) * 2.0 ** -24) + 6 * (n / 4 + 32) * 2.0 ** -33
    off = np.max(np.abs(got[others:, 0] - want), axis=0)
    print("peak", n, rows, D, gap, np.max(off / tol), np.max(off[1:] / mass[1:]), flush=True)
    assert np.all(off <= tol)


@pytest.mark.parametrize("width", [2, 64])
def test_no_rows_a_sequence(torch, width):
    # max_q 0, as the largest row count of a batch without new rows gives it; also inside a capture
    dev, i32 = B.KV4Cache.empty(4, 2, 64, 64), dict(dtype=torch.int32, device="cuda")
    batch = B.KVBatch(torch.zeros(3, width, **i32), torch.full((3,), 40, **i32), torch.zeros(4, **i32), rows=5, max_q=0)
    q, o = torch.ones(5, 4, 64, device="cuda"), torch.full((5, 4, 64), 7.0, device="cuda")
    assert B.attn_kv4(dev, batch, q, 0.1, o=o) is o
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o.add_(1)
        B.attn_kv4(dev, batch, q, 0.1, o=o)
    g.replay()
    torch.cuda.synchronize()
    assert bool((o == 8).all())


def run_cut(torch, new, ctx, heads, G, D, page, dtype, causal=True, window=0, seed=0, edit=None, max_q=None, width=None):
    """As run, over contexts so long that they are cut and joined (random codes, scales past a length stale)."""
    print("cut", new[:6], ctx[:6], heads, G, D, dtype, causal, window, flush=True)
    rng = np.random.default_rng(seed)
    start, seq_len = C.ragged(new), np.array(new) + np.array(ctx)
    T = int(start[-1]) + 2
    table, pages = C.page_table(rng, seq_len, page, width)
    ref = O.Cache(pages, heads, page, D, rng)
    for b, n in enumerate(seq_len):
        for j in range((int(n) + page - 1) // page):
            m = min(int(n) - j * page, page)
            ref.k_scale[table[b, j], :, :m] = 0.35 * np.exp(rng.uniform(-0.5, 0.5, (heads, m)))
            ref.v_scale[table[b, j], :, :m] = 0.4 * np.exp(rng.uniform(-1, 1, (heads, m)))
    if edit is not None:
        edit(table, pages)
    q = O.to_dtype(1.5 * rng.standard_normal((T, heads * G, D)), dtype)
    cache, batch = C.device_cache(torch, ref), C.device_batch(torch, table, seq_len, start, T, max_q or max(new))
    assert B.attn_kv4_workspace(cache, batch, heads * G, C.torch_dtype(torch, dtype)) > 0, "not cut"
    o = torch.full(q.shape, 33.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    B.attn_kv4(cache, batch, C.put(torch, q, dtype), D ** -0.5, causal=causal, window=window, o=o)
    got = C.host(o)
    assert np.all(got[start[-1]:] == 33.0), "padding rows were written"
    want, mass, reach = O.attention(q, ref, table, seq_len, start, D ** -0.5, causal, window)
    n = start[-1]
    off, tol = np.abs(got - want)[:n], C.attention_tolerance(dtype, want[:n], mass[:n], reach[:n], int(seq_len.max()))
    assert np.all(off <= tol), "off by %g of the tolerance at %s" % (np.max(off / tol), np.unravel_index(np.argmax(off / tol), off.shape))


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1500), (False, 4300)])
@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D,G,page", [(64, 8, 32), (128, 5, 64), (256, 3, 128)])
def test_cut_contexts_of_blocks(torch, D, G, page, dtype, causal, window):
    # tiles of 32 columns (16 where D is 256), with rows that see nothing of a part, and a sequence without rows
    run_cut(torch, [16, 5, 0, 16, 1], [5003, 4100, 700, 30, 1999], 2, G, D, page, dtype, causal, window, seed=D + window)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D,G", [(64, 5), (128, 5), (256, 7), (128, 2), (64, 1)])
def test_cut_contexts_of_few_pairs(torch, D, G, dtype):
    # 9 to 16 (row, head) pairs of a KV head: one tile of 16 columns, f32 in two products; and up to 8
    run_cut(torch, [3 if G == 5 else 2, 1, 2], [6001, 90, 2500], 2, G, D, 64, dtype, seed=D + G)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D,G,n,ctx,causal,window", [(128, 5, 300, 4500, True, 0), (64, 8, 300, 4500, False, 0), (256, 3, 300, 4500, True, 0),
                                                     (128, 5, 1200, 4800, True, 0), (128, 5, 1200, 3800, True, 2000), (64, 4, 4300, 0, True, 0)])
def test_cut_contexts_of_prompts(torch, D, G, n, ctx, causal, window, dtype):
    # many tiles in a few parts each, the early ones of a causal prompt in fewer; the join takes several columns a
    # workgroup, a number that does not divide its threads
    run_cut(torch, [n, 7], [ctx, 2000], 2 if n < 1000 else 1, G, D, 64, dtype, causal, window, seed=n + D)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("nseq,heads,G,D,most", [(65, 2, 5, 128, 1), (200, 8, 5, 128, 1), (100, 4, 8, 64, 1), (130, 2, 4, 256, 2), (512, 1, 3, 64, 1),
                                                 (100, 2, 5, 128, 16)])
def test_cut_contexts_of_many_sequences(torch, nseq, heads, G, D, most, dtype):
    # more than the 64 sequences that a wave looks at at once: sums over them run on, few contexts are long
    rng = np.random.default_rng(nseq)
    ctx = rng.integers(0, 300, nseq)
    ctx[[3, 64, nseq - 1]] = [9000, 5111, 4700]
    new = np.full(nseq, most) if most == 1 else rng.integers(0, most + 1, nseq)
    new[[3, 64, nseq - 1]] = most
    run_cut(torch, list(new), list(ctx), heads, G, D, 64, dtype, seed=nseq + D, max_q=most)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cut_contexts_with_absent_pages(torch, dtype):
    def edit(table, pages):
        table[0, 5:60] = -1                                    # a hole over whole parts
        table[1, 0], table[1, 33] = pages, -9
        table[2, :] = -1                                       # nothing is left: zeros
    for new in ([1, 1, 1], [16, 16, 16], [200, 3, 40]):
        run_cut(torch, new, [5000, 4800, 4500], 2, 5, 128, 64, dtype, seed=sum(new), edit=edit)


def test_a_cut_context_of_many_heads_and_a_wide_table(torch):
    # 40 heads on one KV head: two tiles a row; a table far wider than the sequences need
    run_cut(torch, [1, 1], [3000, 77], 1, 40, 128, 64, "bf16", seed=1, width=3000)
    run_cut(torch, [1, 1], [900, 77], 2, 5, 64, 32, "f32", seed=2, width=6000)


def test_rows_past_max_q_of_a_cut_context(torch):
    rng = np.random.default_rng(22)
    ref = O.Cache(100, 2, 64, 128, rng)
    ref.k_scale[:], ref.v_scale[:] = np.float16(0.2), np.float16(0.3)
    table, n, rows = rng.permutation(100).astype(np.int32)[None], 6100, 20
    q = rng.standard_normal((rows, 10, 128)).astype(np.float32)
    batch = C.device_batch(torch, table, [n], C.ragged([rows]), rows, max_q=7)
    dev, o = C.device_cache(torch, ref), torch.full((rows, 10, 128), 5.0, device="cuda")
    assert B.attn_kv4_workspace(dev, batch, 10, torch.float32) > 0
    got = C.host(B.attn_kv4(dev, batch, C.put(torch, q), 0.1, o=o))
    want, mass, reach = O.attention(q, ref, table, np.array([n]), C.ragged([rows]), 0.1, True, 0)
    assert np.all(got[7:] == 5)
    assert np.all(np.abs(got - want)[:7] <= C.attention_tolerance("f32", want, mass, reach, n)[:7])


@pytest.mark.parametrize("dtype,q_size,sm", [("f32", 1e36, 1.0), ("f32", 1e30, 2.0 ** 60), ("bf16", 1e37, 0.5), ("f32", 1.0, 2.0 ** 126),
                                             ("f16", 3.0, 2.0 ** 126), ("f32", 1e-30, 2.0 ** 126), ("bf16", 1e20, 1e20)])
@pytest.mark.parametrize("n,ctx", [(1, 60), (12, 60), (40, 1100)])
def test_scores_past_f32(torch, n, ctx, dtype, q_size, sm):
    """Scores of more than 2^128: all of a row goes to its largest score, wherever that is ahead of the next by more
    than the products' rounding (2^-14 of the largest sum of magnitudes, far more than they lose).  Its weight, 1, is held
    in two f16 parts (2^-21) or one (2^-11), the quotient and the output round."""
    rng = np.random.default_rng(n)
    H, G, D, page, total = 1, 1, 64, 32, n + ctx
    ref = O.Cache((total + page - 1) // page, H, page, D, rng)
    table = rng.permutation(ref.pages).astype(np.int32)[None]
    C.fill_cache(rng, ref, table, [total])
    q = O.to_dtype(q_size * rng.standard_normal((n, H * G, D)), dtype)
    got = C.host(B.attn_kv4(C.device_cache(torch, ref), C.device_batch(torch, table, [total], C.ragged([n]), n),
                            C.put(torch, q, dtype), sm))
    K, V, _ = O.tokens_of(ref, table[0], total)
    clear = 0
    for i in range(n):
        k, v = K[:ctx + i + 1, 0], V[:ctx + i + 1, 0]
        score = k @ q[i, 0].astype(np.float64)
        first, second = np.argsort(score)[[-1, -2]]
        reach = np.max(np.abs(k) @ np.abs(q[i, 0].astype(np.float64)))
        if score[first] - score[second] < 2.0 ** -13 * reach or (score[first] - score[second]) * sm < 1000:
            continue
        clear += 1
        want = v[first]
        assert np.all(np.abs(got[i, 0] - want) <= np.abs(want) * ((2.0 ** -21 if dtype == "f32" else 2.0 ** -11) + 2.0 ** -22 + O.EPS[dtype] / 2)
                      + 2.0 ** -25), i
    assert clear >= (n + 1) // 2
