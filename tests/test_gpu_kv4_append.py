"""GPU: rad_kv4_append and rad_kv4_read against the oracle: codes, scales, turned queries (f32) and the read-back bit
for bit; everything that the call does not append to stays as it was."""
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


def bits(t):
    return t.cpu().contiguous().view(__import__("torch").uint8).numpy()


def run(torch, new, ctx, heads, q_heads, D, page, dtype, rope=None, style=0, rot=False, seed=0, pad=0, table_edit=None,
        with_q=True, fused=True, rope_rows=None):
    """One append against the oracle, then the read-back.  `new`, `ctx`: tokens appended and already there."""
    rng = np.random.default_rng(seed)
    start = C.ragged(new)
    T = int(start[-1]) + pad
    seq_len = np.array(new) + np.array(ctx)
    table, pages = C.page_table(rng, np.maximum(seq_len, 0), page)
    if table_edit is not None:
        table_edit(table, pages)
    ref = O.Cache(pages, heads, page, D, rng)
    dev = C.device_cache(torch, ref)
    x = rng.standard_normal((T, q_heads + 2 * heads, D)) * np.exp(rng.uniform(-4, 4, (T, q_heads + 2 * heads, 1)))
    x[..., 5] *= 9
    x = O.to_dtype(x, dtype)
    tab = None if rope is None else C.rope_table(int(max(seq_len.max(), 1)) if rope_rows is None else rope_rows, rope)
    xd = C.put(torch, x, dtype)
    qd, kd, vd = xd.split([q_heads, heads, heads], dim=1)
    if not fused:
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    one = all(n == 1 for n in new) and pad == 0
    batch = C.device_batch(torch, table, seq_len, None if one else start, T)
    q_out = torch.full((T, q_heads, D), 77.0, dtype=C.torch_dtype(torch, dtype), device="cuda") if with_q else None
    out = B.kv4_append(dev, batch, kd, vd, qd if with_q else None, rope=None if tab is None else C.put(torch, tab),
                       rope_style=style, rotate=rot, q_out=q_out)
    ko, vo = (torch.full((T, heads, D), 55.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.kv4_read(dev, batch, ko, vo)
    torch.cuda.synchronize()

    q_ref = np.full((T, q_heads, D), 77.0, np.float32)
    k_ref, v_ref = np.full((T, heads, D), 55.0), np.full((T, heads, D), 55.0)
    for b, n in enumerate(new):
        for i in range(n):
            row, pos = int(start[b]) + i, int(seq_len[b]) - n + i
            if pos < 0:
                continue
            skip = tab is not None and pos >= len(tab)
            page_id = int(table[b, pos // page])
            if not skip:
                q1, k1, v1 = O.append_f32(x[row:row + 1, :q_heads], x[row:row + 1, q_heads:q_heads + heads],
                                          x[row:row + 1, q_heads + heads:], None if tab is None else tab[pos:pos + 1],
                                          style, rot)
                q_ref[row] = O.to_dtype(q1[0], dtype)
                if 0 <= page_id < pages:
                    ref.put(page_id, pos % page, (k1[0][0], k1[1][0]), (v1[0][0], v1[1][0]))
            if 0 <= page_id < pages:
                k_ref[row], v_ref[row] = ref.get(page_id, pos % page)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        got, want = bits(getattr(dev, name)), getattr(ref, name).view(np.uint8).reshape(bits(getattr(dev, name)).shape)
        assert np.array_equal(got, want), "%s differs in %d bytes" % (name, np.count_nonzero(got != want))
    if with_q:
        assert out is q_out and np.array_equal(C.host(q_out), q_ref)
    assert np.array_equal(C.host(ko), O.bf16_round(k_ref.astype(np.float32)), equal_nan=True)
    assert np.array_equal(C.host(vo), O.bf16_round(v_ref.astype(np.float32)), equal_nan=True)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("D,rope,style,rot", [(128, 128, 0, True), (128, 64, 1, True), (128, 64, 0, False), (256, 256, 0, True),
                                              (256, 128, 1, True), (64, 64, 0, False), (64, 24, 1, False), (64, 8, 0, False),
                                              (128, None, 0, True), (128, None, 0, False)])
def test_decode_and_blocks(torch, D, rope, style, rot, dtype):
    print("append", D, rope, style, rot, dtype, flush=True)
    run(torch, [1, 1, 1], [0, 31, 70], 2, 6, D, 32, dtype, rope, style, rot, seed=D)                # one token each
    run(torch, [5, 0, 16, 3], [3, 9, 62, 0], 3, 5 * 3, D, 64, dtype, rope, style, rot, seed=D + 1)  # ragged, odd
    run(torch, [1], [0], 1, 1, D, 32, dtype, rope, style, rot, seed=D + 2)


@pytest.mark.parametrize("page", B.KV4_PAGE_SIZES)
@pytest.mark.parametrize("ctx", [0, 1, 7, 8, 37, 250])
def test_prompts_of_many_rows(torch, page, ctx):
    # a workgroup walks eight rows
    print("append prompt", page, ctx, flush=True)
    run(torch, [600, 0, 1, 13], [ctx, 5, 40, 2 * ctx], 1, 2, 64, page, "f32", 64, 0, False, seed=page + ctx)


def test_padding_rows_and_separate_arrays(torch):
    run(torch, [3, 2], [4, 30], 2, 4, 128, 32, "bf16", 128, 0, True, pad=6)
    run(torch, [3, 2], [4, 30], 2, 4, 128, 32, "f32", 128, 0, True, fused=False)
    run(torch, [3, 2], [4, 30], 2, 4, 128, 32, "f16", 128, 0, True, with_q=False)


@pytest.mark.parametrize("D,rot", [(64, False), (128, True), (256, True)])
def test_one_row_each_of_many_sequences(torch, D, rot):
    # lengths around octets and pages, no token at all, an absent page, a position past the table
    def edit(table, pages):
        table[5, -1] = -1
        table[40] = -1
    rng = np.random.default_rng(D)
    ctx = rng.integers(0, 70, 90)
    ctx[:9] = [-1, 0, 6, 7, 8, 64, 31, 32, 95]
    print("append one row each", D, flush=True)
    run(torch, [1] * 90, ctx, 2, 3, D, 32, "bf16", D // 2, 0, rot, table_edit=edit, rope_rows=95)
    run(torch, [1] * 90, ctx, 2, 3, D, 32, "f32", D, 1, rot, with_q=False)


@pytest.mark.parametrize("new", [[2, 3, 2], [4, 5, 6, 1], [1, 0, 9, 0, 30, 2], [3] * 70, [17, 16, 15] * 30])
def test_blocks_of_every_size(torch, new):
    # rows a workgroup go by the rows a sequence has on average: 2, 4, 8
    print("append blocks", len(new), new[:6], flush=True)
    rng = np.random.default_rng(len(new))
    run(torch, new, rng.integers(0, 40, len(new)), 2, 3, 128, 32, "f16", 128, 0, True, pad=1)


def test_absent_pages_and_rows_before_the_first_token(torch):
    def edit(table, pages):
        table[0, 1] = -1
        table[1, 0] = pages                                    # past the pool
        table[2, 0] = 2 ** 31 - 1
    run(torch, [40, 5, 3], [20, 0, 1], 2, 2, 64, 32, "f32", 64, 0, False, table_edit=edit)
    run(torch, [6, 4], [-2, 3], 2, 2, 64, 32, "f32", 64, 0, False)     # seq_len below the rows: two rows are no token


def test_positions_past_the_table_are_skipped(torch):
    run(torch, [20, 3], [10, 27], 2, 2, 128, 32, "f32", 128, 0, True, rope_rows=25)


def test_zero_vectors_and_extreme_scales(torch):
    rng = np.random.default_rng(3)
    ref = O.Cache(1, 1, 32, 64)
    dev = C.device_cache(torch, ref)
    x = np.zeros((8, 1, 64), np.float32)
    x[1, 0, 3] = 1e-7                                          # scale is a subnormal f16
    x[2, 0, 3] = 1e-12                                         # scale rounds to zero
    x[3] = rng.standard_normal((1, 64)) * 1e6                  # scale saturates
    x[4, 0] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 8) * np.where(np.arange(64) % 3, 1, -1)   # ties
    x[5, 0, 0] = 3.0e38
    x[6] = -0.0
    x[7] = rng.standard_normal((1, 64))
    batch = C.device_batch(torch, np.zeros((1, 1), np.int32), [8], C.ragged([8]), 8)
    B.kv4_append(dev, batch, C.put(torch, x), C.put(torch, x), rotate=False)
    for t in range(8):
        kc, s = O.quantise_f32(x[t])
        ref.put(0, t, (kc, s), (kc, s))
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert np.array_equal(bits(getattr(dev, name)).ravel(), getattr(ref, name).view(np.uint8).ravel()), name


def test_every_tie_and_its_neighbours(torch):
    # with a largest value of 6 the scale is 1 and the quotients are the values themselves
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(9)), np.nextafter(mids, np.float32(0)), O.LEVELS[1:7]])
    v = np.concatenate([v, -v]).astype(np.float32)
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :len(v)], x[0, 0, 63] = v, 6.0
    assert len(v) < 63
    dev = C.device_cache(torch, O.Cache(1, 1, 32, 64))
    batch = C.device_batch(torch, np.zeros((1, 1), np.int32), [1], None, 1)
    B.kv4_append(dev, batch, C.put(torch, x), C.put(torch, x), rotate=False)
    kc = dev.k_codes.cpu().numpy()[0, 0, 0]
    got = np.stack([kc & 15, kc >> 4], axis=1).ravel()
    assert np.array_equal(got, O.e2m1_codes(x[0, 0]))


def test_appending_token_by_token_equals_appending_at_once(torch):
    rng = np.random.default_rng(9)
    n, H, D, page = 45, 2, 128, 32
    x = C.put(torch, rng.standard_normal((n, 3 * H, D)).astype(np.float32))
    table = np.array([[1, 0]], np.int32)
    tab = C.put(torch, C.rope_table(64, 128))
    once, steps = (C.device_cache(torch, O.Cache(2, H, page, D)) for _ in range(2))
    q, k, v = x.split([H, H, H], dim=1)
    whole = B.kv4_append(once, C.device_batch(torch, table, [n], C.ragged([n]), n), k, v, q, rope=tab)
    for t in range(n):
        one = B.kv4_append(steps, C.device_batch(torch, table, [t + 1], None, 1), k[t:t + 1], v[t:t + 1], q[t:t + 1],
                           rope=tab)
        assert torch.equal(one[0], whole[t])
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert np.array_equal(bits(getattr(once, name)), bits(getattr(steps, name))), name


def test_binding_refusals(torch):
    dev = B.KV4Cache.empty(2, 2, 32, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = B.KVBatch(torch.zeros(1, 1, **i32), torch.ones(1, **i32), torch.zeros(2, **i32), rows=3)
    k = torch.zeros(3, 2, 64, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        B.kv4_append(dev, batch, k[:2], k)
    with pytest.raises(TypeError, match="v must be"):
        B.kv4_append(dev, batch, k, k.half())
    with pytest.raises(ValueError, match="contiguous"):
        B.kv4_append(dev, batch, torch.zeros(3, 64, 2, device="cuda").transpose(1, 2), k)
    with pytest.raises(B.RadError):
        B.kv4_append(dev, batch, k, k, rotate=True)            # 64 values a head: no rotation
    with pytest.raises(ValueError, match="q_out"):
        B.kv4_append(dev, batch, k, k, q_out=k, rotate=False)
    with pytest.raises(B.RadError):
        B.kv4_append(dev, batch, k[:1].expand(3, 2, 64), k, rotate=False)   # rows on top of each other
    with pytest.raises(ValueError, match="rows"):
        B.KVBatch(torch.zeros(1, 1, **i32), torch.ones(1, **i32), torch.zeros(2, **i32))
    with pytest.raises(ValueError, match="page size"):
        B.KV4Cache.empty(2, 2, 48, 64)
    with pytest.raises(ValueError, match="v_scale"):
        B.KV4Cache(dev.k_codes, dev.k_scale, dev.v_codes, dev.v_scale[:1])


@pytest.mark.parametrize("D,heads,q_heads,new,dtype,rope,style,rot", [
    (256, 3, 9, [2000, 0, 1, 1500, 33, 466], "bf16", 256, 0, True),       # seven groups of heads a workgroup, three workgroups a row
    (256, 3, 9, [1200, 900], "f32", 128, 1, False),                       # three groups a workgroup
    (128, 4, 20, [3000, 9, 700, 491], "f32", 128, 0, True),               # seven groups of two heads
    (128, 4, 19, [2500, 17, 60], "f16", 64, 1, True),                     # five, the last with one head to spare
    (128, 4, 20, [3000, 9, 700, 491], "bf16", None, 0, False),
    (64, 4, 20, [9001], "f16", 64, 0, False),                             # seven groups of four heads, all of a row's
    (64, 5, 17, [2400, 2403], "f32", 24, 1, False)])
def test_prompts_whose_workgroups_take_several_groups_of_heads(torch, D, heads, q_heads, new, dtype, rope, style, rot):
    print("append groups", D, heads, q_heads, new, dtype, flush=True)
    rng = np.random.default_rng(D + heads)

    def edit(table, pages):
        table[0, 3] = -1
    run(torch, new, rng.integers(0, 50, len(new)), heads, q_heads, D, 64, dtype, rope, style, rot, pad=3, table_edit=edit)
