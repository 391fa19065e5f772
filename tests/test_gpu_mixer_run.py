"""GPU: the token mixers used together, as a serving program does: trees drafted, verified and their accepted path kept;
a session whose cache is cut by weight and goes on; linear attention between rotated linears; captured graphs whose
inputs move on; several streams at once; caches and states past 2^32 bytes."""
import numpy as np
import pytest

import layer_cases as C
from oracle import layer as O
from oracle import mixers as X
from rotated_w8a8_int8_amd import binding as B
from test_gpu_layer_run import linear_within_quantisation, weight

pytestmark = pytest.mark.gpu
REPLAYS = 4
ARRAYS = ("k_codes", "v_codes", "k_scale", "v_scale")


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def i32(torch, a):
    return C.put(torch, np.asarray(a, np.int32))


def host_cache(cache):
    c = O.Cache(cache.pages, cache.heads, cache.page_size, cache.D)
    for name in ARRAYS:
        getattr(c, name)[:] = getattr(cache, name).cpu().numpy()
    return c


@pytest.mark.parametrize("dtype,D,style", [("f32", 128, 0), ("bf16", 128, 1), ("f16", 64, 0)])
def test_trees_are_verified_and_their_path_kept(torch, dtype, D, style):
    # two sequences draft a tree three times; the path accepted is what appending it alone would have left
    rng = np.random.default_rng(D + style)
    H, G, page, width, rot = 2, 3, 32, 6, D % 128 == 0
    tab = C.put(torch, C.rope_table(width * page, D))
    host = O.Cache(2 * width, H, page, D, rng)
    table = np.arange(2 * width, dtype=np.int32).reshape(2, width)
    C.fill_cache(rng, host, table, [40, 61], k_size=10.0 if rot else 1.0)
    cache, plain = C.device_cache(torch, host), C.device_cache(torch, host)
    lens = np.array([40, 61])
    for _ in range(3):
        n = 20
        parents = [[-1] + [int(rng.integers(max(-1, i - 4), i)) for i in range(1, n)] for _ in range(2)]
        masks, depth = np.zeros((2, n), np.uint64), np.zeros((2, n), np.int64)
        for b in range(2):
            for i, p in enumerate(parents[b]):
                masks[b, i] = (masks[b, p] if p >= 0 else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
                depth[b, i] = depth[b, p] + 1 if p >= 0 else 0
        x = O.to_dtype(rng.standard_normal((2 * n, H * G + 2 * H, D)), dtype)
        q, k, v = C.put(torch, x, dtype).split([H * G, H, H], dim=1)
        batch = C.device_batch(torch, table, lens + n, C.ragged([n, n]), 2 * n, n)
        where = i32(torch, (lens[:, None] + depth).reshape(-1))
        qt = B.kv4_append(cache, batch, k, v, q, rope=tab, rope_style=style, rotate=rot, position=where)
        mask = C.put(torch, masks.reshape(-1, 1).view(np.int64))
        o = B.attn_kv4_tree(cache, batch, qt, mask, sm_scale=D ** -0.5)
        want, mass, reach, _ = X.attend(C.host(qt), host_cache(cache), table, lens + n, C.ragged([n, n]), D ** -0.5,
                                        lambda b, m, L, on: X.sees_tree(m, L, on, masks[b][:, None], 0))
        assert np.all(np.abs(C.host(o) - want) <= C.attention_tolerance(dtype, want, mass, reach, int(lens.max()) + n))
        # accept a path from the root of each: the longest, and a random one of three nodes at most
        paths = []
        for b in range(2):
            node, path = (int(np.argmax(depth[b])) if b == 0 else int(rng.integers(0, n))), []
            while node >= 0:
                path.append(node)
                node = parents[b][node]
            paths.append(path[::-1][:9 if b == 0 else 3])
        kept, src = [len(p) for p in paths], np.full((2, 9), -1, np.int32)
        for b, p in enumerate(paths):
            src[b, :len(p)] = lens[b] + np.array(p)
        B.kv4_move(cache, batch, i32(torch, src), i32(torch, kept), to_start=i32(torch, lens))
        # the same tokens as a chain
        rows = torch.tensor([b * n + i for b in range(2) for i in paths[b]], device="cuda")
        chain = C.device_batch(torch, table, lens + kept, C.ragged(kept), sum(kept))
        B.kv4_append(plain, chain, k[rows], v[rows], q[rows], rope=tab, rope_style=style, rotate=rot)
        lens = lens + kept
        a, b_ = host_cache(cache), host_cache(plain)
        for s in range(2):
            for got, want in zip(O.tokens_of(a, table[s], int(lens[s])), O.tokens_of(b_, table[s], int(lens[s]))):
                assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_session_is_cut_by_weight_and_goes_on(torch, dtype):
    rng = np.random.default_rng(5)
    H, G, D, page, budget, width = 2, 4, 64, 32, 64, 8
    ctx = [150, 40]
    table, pages = C.page_table(rng, np.array([width * page] * 2), page)
    host = O.Cache(pages, H, page, D, rng)
    cache = C.device_cache(torch, host)
    tab = C.put(torch, C.rope_table(400, D))
    sm = D ** -0.5

    def draw(n):
        return O.to_dtype(rng.standard_normal((n, H * G + 2 * H, D)), dtype)
    # prompts, observed from their last 16 rows
    x = draw(sum(ctx))
    q, k, v = C.put(torch, x, dtype).split([H * G, H, H], dim=1)
    batch = C.device_batch(torch, table, ctx, C.ragged(ctx), sum(ctx))
    qt = B.kv4_append(cache, batch, k, v, q, rope=tab, rotate=False)
    w = torch.full((2, H, width * page), float("nan"), device="cuda")
    B.attn_kv4_weights(cache, batch, qt, w, sm, observe=16, factor=0.0)
    total = w.clone()
    # three tokens, their weights added
    lens = np.array(ctx)
    for _ in range(3):
        lens = lens + 1
        q, k, v = C.put(torch, draw(2), dtype).split([H * G, H, H], dim=1)
        one = C.device_batch(torch, table, lens, None, 2)
        qt = B.kv4_append(cache, one, k, v, q, rope=tab, rotate=False)
        B.attn_kv4_weights(cache, one, qt, w, sm)
        assert torch.all(torch.nan_to_num(w) >= torch.nan_to_num(total))
        total = w.clone()
    for b, n in enumerate(ctx):                              # 16 rows and 3 tokens of G heads each
        assert abs(float(w[b, :, :lens[b]].sum()) - H * G * (16 + 3)) < 1e-3
    # the cut: exactly what the weights say, to new pages
    one = C.device_batch(torch, table, lens, None, 2)
    kept, count, kw = B.kv4_select(one, w, budget, first=2, recent=8)
    to_table, to_pages = C.page_table(rng, np.array([width * page] * 2), page)
    small = B.KV4Cache.empty(to_pages, H, page, D)
    B.kv4_move(cache, one, kept, count, to=small, to_table=C.put(torch, to_table))
    before, after = host_cache(cache), host_cache(small)
    for b in range(2):
        K, V, _ = O.tokens_of(before, table[b], int(lens[b]))
        k2, v2, _ = O.tokens_of(after, to_table[b], min(budget, int(lens[b])))
        for h in range(H):
            at = X.select(w[b, h].cpu().numpy(), int(lens[b]), budget, 2, 8)
            assert np.array_equal(kept[b, h, :len(at)].cpu().numpy(), at)
            assert np.array_equal(k2[:, h], K[at, h]) and np.array_equal(v2[:, h], V[at, h])
    # it goes on: places in the cache and positions have parted
    new_len = np.minimum(lens, budget)
    w2 = torch.zeros((2, H, width * page), device="cuda")
    w2[:, :, :kw.shape[2]] = kw
    for _ in range(2):
        lens, new_len = lens + 1, new_len + 1
        q, k, v = C.put(torch, draw(2), dtype).split([H * G, H, H], dim=1)
        one = C.device_batch(torch, to_table, new_len, None, 2)
        qt = B.kv4_append(small, one, k, v, q, rope=tab, rotate=False, position=i32(torch, lens - 1))
        turned = O.turn_f32(C.host(q), C.rope_table(400, D)[lens - 1], 0)
        assert np.array_equal(C.host(qt), O.to_dtype(turned, dtype))
        o, _ = B.attn_kv4_weights(small, one, qt, w2, sm, factor=0.5)
        want, mass, reach, _ = X.attend(C.host(qt), host_cache(small), to_table, new_len, C.ragged([1, 1]), sm,
                                        lambda b, n, m, on: X.sees_position(n, m, on, True, 0))
        assert np.all(np.abs(C.host(o) - want) <= C.attention_tolerance(dtype, want, mass, reach, 300))


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 3, 100]])
def test_linear_attention_between_linears(torch, new):
    # norm, fused projection, mixer, output projection: each step from what the one before left
    hidden, H, D, T, rng = 512, 4, 64, sum(new), np.random.default_rng(3)
    wq, wq_values = weight(torch, hidden, 3 * H * D, 5)
    wo, wo_values = weight(torch, H * D, hidden, 6)
    gamma = C.put(torch, np.ones(hidden, np.float32))
    x = rng.standard_normal((T, hidden)).astype(np.float32)
    q8, s8, _ = B.add_rmsnorm_quant_i8(C.put(torch, x), gamma)
    contract = B.w8a8_gemv if T <= B.RAD_GEMV_MAX_M else B.w8a8_gemm
    y = contract(q8, s8, wq)[0]
    q, k, v = y.view(T, 3 * H, D).split([H, H, H], dim=1)
    g = -np.exp2(-np.arange(1, H + 1)).astype(np.float32)
    start = C.ragged(new)
    s0 = rng.standard_normal((3, H, D, D)).astype(np.float32)
    state = C.put(torch, s0)
    o, _ = B.linear_attn(q, k, v, C.put(torch, g), state=state, state_out=state, q_start=None if max(new) == 1 else C.put(torch, start),
                         max_q=max(new), scale=D ** -0.5)
    o8, t8 = B.quant_act_i8(o.view(T, H * D), rotate=True)
    z = contract(o8, t8, wo)[0]
    _, n, _ = O.add_rmsnorm(x, None, np.ones(hidden), 1e-6, "f32", True)
    linear_within_quantisation(y.cpu().numpy(), n, wq_values, s8.cpu().numpy().astype(np.float64))
    yq = y.cpu().numpy().reshape(T, 3 * H, D)
    want, S, mass, big = X.linear(yq[:, :H], yq[:, H:2 * H], yq[:, 2 * H:], g, s0, start, D ** -0.5)
    f32 = (6 * max(new) + D + 128) * 2.0 ** -24                 # as in test_gpu_linear_attn.tolerance
    assert np.all(np.abs(C.host(o) - want) <= f32 * mass + 2.0 ** -24 * np.abs(want) + 1e-30)
    assert np.all(np.abs(state.cpu().numpy() - S) <= f32 * big + 1e-30)
    linear_within_quantisation(z.cpu().numpy(), O.rotate(o.cpu().numpy().reshape(T, -1)), wo_values, t8.cpu().numpy().astype(np.float64))


def replay(torch, step, outs, inputs, change, scratch):
    """Captures step, and replays it REPLAYS times after `change`, its scratch full of NaN, against the eager step on the
    same inputs (`inputs` are what it updates in place)."""
    def bits():
        return [t.view(torch.uint8).clone() for t in outs + inputs]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(REPLAYS):
        change(r)
        torch.cuda.synchronize()
        saved = [t.clone() for t in inputs]
        step()
        torch.cuda.synchronize()
        want = bits()
        for t, s in zip(inputs, saved):
            t.copy_(s)
        for t in outs:
            t.view(torch.uint8).fill_(255)
        for t in scratch:
            t.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(bits(), want)):
            assert torch.equal(a, b), "replay %d: output %d differs" % (r, i)


@pytest.mark.parametrize("n,dtype,cap", [(1, "f32", 200), (7, "bf16", 3000), (1, "f16", 70000)])
def test_graph_replays_of_a_session(torch, n, dtype, cap):
    # attention with weights, selection (in slices for the longest) and move, lengths and table changing between replays
    rng = np.random.default_rng(n + cap)
    H, G, D, page, B_, budget = 2, 4, 64, 64, 2, 48
    width = (cap + page - 1) // page
    host = O.Cache(B_ * width, H, page, D, rng)
    host.k_scale[:], host.v_scale[:] = np.float16(0.2), np.float16(0.4)
    cache, dt = C.device_cache(torch, host), C.torch_dtype(torch, dtype)
    table = C.put(torch, rng.permutation(B_ * width).reshape(B_, width).astype(np.int32))
    lens = i32(torch, [cap // 2, cap // 3])
    batch = B.KVBatch(table, lens, None if n == 1 else C.put(torch, C.ragged([n] * B_)), rows=B_ * n, max_q=n)
    q = torch.randn((B_ * n, H * G, D), device="cuda").to(dt)
    w = torch.rand((B_, H, width * page), device="cuda")
    to = B.KV4Cache.empty(2 * B_, H, 32, D)
    to_table = i32(torch, np.arange(2 * B_).reshape(B_, 2))
    mask = torch.full((B_ * n, 1), 5, dtype=torch.int64, device="cuda")
    o, ot, kept, count = torch.empty_like(q), torch.empty_like(q), torch.empty((B_, H, budget), dtype=torch.int32, device="cuda"), i32(torch, [0, 0])
    kw = torch.empty((B_, H, budget), device="cuda")
    scratch = [torch.empty(max(k, 16), dtype=torch.uint8, device="cuda") for k in (
        B.attn_kv4_weights_workspace(cache, batch, H * G, dt), B.attn_kv4_workspace(cache, batch, H * G, dt),
        B.kv4_select_workspace(B_, H, width * page))]
    assert (B.kv4_select_workspace(B_, H, width * page) > 0) == (cap > 65536)

    def step():
        B.attn_kv4_weights(cache, batch, q, w, 0.1, factor=0.5, o=o, workspace=scratch[0])
        B.attn_kv4_tree(cache, batch, q, mask, 0.1, o=ot, workspace=scratch[1])
        B.kv4_select(batch, w, budget, 3, 9, kept=kept, count=count, kept_weight=kw, workspace=scratch[2])
        B.kv4_move(cache, batch, kept, count, to=to, to_table=to_table)

    def change(r):
        lens.copy_(torch.tensor([[cap - 3, 20], [5, cap // 2], [cap, cap], [60, 0]][r], dtype=torch.int32))
        table.copy_(table.flip(1))
        q.mul_(-1.01)
        mask.add_(2)
        kept.zero_(), kw.zero_()
    # what selection leaves as it was is set again before each of the two
    outs, inputs = [o, ot, count], [w, kept, kw] + [getattr(to, name) for name in ARRAYS]
    replay(torch, step, outs, inputs, change, scratch)


@pytest.mark.parametrize("dtype,n,D", [("bf16", 900, 128), ("f32", 700, 64), ("f16", 3, 128)])
def test_graph_replays_of_linear_attention(torch, dtype, n, D):
    H, dt = 4, C.torch_dtype(torch, dtype)
    qkv = torch.randn((2 * n, 3 * H, D), device="cuda").to(dt)
    q, k, v = qkv.split([H, H, H], dim=1)
    g, state = -torch.rand(H, device="cuda"), torch.randn((2, H, D, D), device="cuda")
    start, o = i32(torch, [0, n, 2 * n]), torch.empty((2 * n, H, D), dtype=dt, device="cuda")
    d = B.LinearDesc(q.data_ptr(), k.data_ptr(), v.data_ptr(), 3 * H * D, 3 * H * D, 3 * H * D, g.data_ptr(), start.data_ptr(), 2, 2 * n,
                     n, H, H, D, {"f32": 0, "bf16": 1, "f16": 2}[dtype])
    import ctypes
    size = ctypes.c_int64(0)
    assert B.lib().rad_linear_attn_workspace(d, ctypes.byref(size)) == B.RAD_OK and (size.value > 0) == (n > 100)
    scratch = torch.empty(max(size.value, 16), dtype=torch.uint8, device="cuda")

    def step():
        B.linear_attn(q, k, v, g, state=state, state_out=state, q_start=start, max_q=n, scale=0.1, o=o, workspace=scratch)

    def change(r):
        qkv.mul_(-0.9)
        g.mul_(0.7)
        start[1] = [n // 3, n, 0, n - 1][r]
        start[2] = [n, 2 * n, n - 2, n][r]
        o.zero_()
    replay(torch, step, [], [state, o], change, [scratch])


def test_several_streams_at_once(torch):
    gen = torch.Generator(device="cuda").manual_seed(4)
    rng = np.random.default_rng(4)
    H, G, D, page, width = 2, 4, 128, 64, 40
    host = O.Cache(2 * width, H, page, D, rng)
    host.k_scale[:], host.v_scale[:] = np.float16(0.2), np.float16(0.4)
    table, cache = np.arange(2 * width, dtype=np.int32).reshape(2, width), C.device_cache(torch, host)
    one = C.device_batch(torch, table, [2500, 700], None, 2)
    many = C.device_batch(torch, table, [2500, 700], C.ragged([60, 40]), 100, 60)
    q1, q2 = torch.randn((2, H * G, D), generator=gen, device="cuda"), torch.randn((100, H * G, D), generator=gen, device="cuda").bfloat16()
    mask = torch.full((100, 1), -1, dtype=torch.int64, device="cuda")
    x = torch.randn((1500, 12, D), generator=gen, device="cuda").bfloat16()
    decay, start = -torch.rand(4, generator=gen, device="cuda"), i32(torch, [0, 900, 1500])
    w = torch.rand((2, H, width * page), generator=gen, device="cuda")
    big = torch.rand((2, H, 80000), generator=gen, device="cuda")
    longs = C.device_batch(torch, np.zeros((2, 1250), np.int32), [80000, 70001], None, 2)

    def jobs():
        yield lambda: B.attn_kv4_weights(cache, one, q1, w.clone(), 0.1)
        yield lambda: B.attn_kv4_weights(cache, many, q2, w.clone(), 0.1, factor=0.5)
        yield lambda: (B.attn_kv4_tree(cache, many, q2, mask, 0.1),)
        yield lambda: B.linear_attn(x[:, :4], x[:, 4:8], x[:, 8:], decay, state_out=torch.zeros((2, 4, D, D), device="cuda"), q_start=start, max_q=900)
        yield lambda: B.kv4_select(longs, big, 3000, 4, 100)[::2]
    want = [[t.clone() for t in job()] for job in jobs()]
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for job, s in zip(jobs(), streams):
            with torch.cuda.stream(s):
                got.append(job())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x_, y_ in zip(a, b):
                assert torch.equal(x_, y_)


def test_caches_and_states_past_32_bits(torch):
    # 34,000 pages of 128 KiB: codes reach past 2^32 bytes; the sequence lies on the first and the last pages
    rng = np.random.default_rng(7)
    pages, H, page, D, n = 34000, 8, 256, 128, 589
    cache, ref = B.KV4Cache.empty(pages, H, page, D), B.KV4Cache.empty(6, H, page, D)
    table, small = np.array([[pages - 1, 0, pages - 2]], np.int32), np.array([[2, 0, 1]], np.int32)
    to_big, to_small = np.array([[pages - 3, 1]], np.int32), np.array([[4, 3]], np.int32)
    x = C.put(torch, rng.standard_normal((n, 3 * H, D)).astype(np.float32))
    q, k, v = x.split([H, H, H], dim=1)
    mask, w0, outs = torch.full((9, 1), 73, dtype=torch.int64, device="cuda"), torch.rand((1, H, 3 * page), device="cuda"), []
    for c, t, to in ((cache, table, to_big), (ref, small, to_small)):
        qo = B.kv4_append(c, C.device_batch(torch, t, [n], C.ragged([n]), n), k, v, q)
        batch = C.device_batch(torch, t, [n], C.ragged([9]), 9, 9)
        o, w = B.attn_kv4_weights(c, batch, qo[-9:].contiguous(), w0.clone(), 0.1)
        kept, count, kw = B.kv4_select(batch, w, 300, 4, 20)
        B.kv4_move(c, batch, kept, count, to_table=C.put(torch, to))
        moved = C.device_batch(torch, to, [300], C.ragged([300]), 300)
        outs.append((o, w, kept, kw, B.attn_kv4_tree(c, batch, qo[-9:].contiguous(), mask, 0.1), *B.kv4_read(c, moved)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    # states of 4.6 GB: the last sequences as they are alone
    del cache, ref, outs
    B_, heads = 1100, 16
    state = torch.empty((B_, heads, 256, 256), device="cuda")
    state[-2:].normal_()
    first = state[-2:].clone()
    q, k, v = (torch.randn((B_, heads, 256), device="cuda").half() for _ in range(3))
    g = -torch.rand(heads, device="cuda")
    o, _ = B.linear_attn(q, k, v, g, state=state, state_out=state)
    o2, s2 = B.linear_attn(q[-2:], k[-2:], v[-2:], g, state=first, state_out=first)
    assert torch.equal(o[-2:], o2) and torch.equal(state[-2:], s2)


def test_unattended_rows_weigh_nothing_and_queries_share_no_scale(torch):
    # rows without a token to see, zero queries and huge ones side by side
    rng = np.random.default_rng(9)
    H, G, D, page = 1, 40, 64, 32
    table, pages = C.page_table(rng, np.array([64]), page)
    host = O.Cache(pages, H, page, D, rng)
    C.fill_cache(rng, host, table, [3])
    q = rng.standard_normal((5, G, D)).astype(np.float32)
    q[2], q[3] = 0.0, q[3] * 1e20
    cache, batch = C.device_cache(torch, host), C.device_batch(torch, table, [3], C.ragged([5]), 5)
    w = torch.zeros((1, H, 64), device="cuda")
    o, _ = B.attn_kv4_weights(cache, batch, C.put(torch, q), w, 1.0, factor=0.0)
    o, w = C.host(o), w.cpu().numpy()[0, 0]
    assert not o[:2].any() and np.isfinite(o).all()              # tokens -2 and -1: none
    assert abs(w.sum() - 3 * G) < 1e-3 and not w[3:].any()
    assert w[0] >= G - 1e-3                                      # the zero query of token 0 sees it alone
