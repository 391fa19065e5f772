"""GPU: the calls between a layer's linears used together, as a decoding program does: norm, fused projection,
append, attention, output projection and the next norm; token by token against all at once; inside captured graphs
whose lengths move on; on two streams at once; in a cache past 2^32 bytes."""
import numpy as np
import pytest

import layer_cases as C
import oracle
from oracle import layer as O
from rotated_w8a8_int8_amd import binding as B
from rotated_w8a8_int8_amd import workloads as W

pytestmark = pytest.mark.gpu
REPLAYS = 4


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


def weight(torch, K, N, seed):
    """Float weights quantised by the library, and their codes times scales in the rotated domain, f64."""
    w = B.quant_weight_i8(torch.from_numpy(W.make_float_weights(N, K, seed=seed)).cuda(), B.RAD_FMT_U8G256_BF16ROW)
    r = W.bf16_bits_to_f32(w.rscale.cpu().numpy().view(np.uint16)).astype(np.float64)
    values = (w.codes.cpu().numpy().astype(np.float64).reshape(N, -1, 256)
              * w.gscale.cpu().numpy().astype(np.float64)[..., None]).reshape(N, K) * r[:, None]
    return w, values


def linear_within_quantisation(y, x_rot, w_values, s):
    """y against x.W^T in f64 from the activations before they were quantised: each code is off by at most half a
    scale, so an output by half a scale times its weights' magnitudes, over 128; and the f32 epilogue, 2^-15 of the
    products' magnitudes."""
    want = x_rot @ w_values.T / 128
    mass = np.abs(w_values).sum(axis=1) / 128
    bound = s[:, None] * mass * (0.5 + 2.0 ** -10) + 2.0 ** -15 * (np.abs(x_rot) @ np.abs(w_values).T) / 128
    assert np.all(np.abs(y - want) <= bound)


@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [40, 0, 95]), ([5, 1, 16], [33, 64, 7]), ([150], [20])])
def test_one_attention_block(torch, new, ctx):
    hidden, H, G, D, page = 512, 2, 2, 128, 32
    HQ, T = H * G, sum(new)
    rng = np.random.default_rng(T)
    start, seq_len = C.ragged(new), np.array(new) + np.array(ctx)
    table, pages = C.page_table(rng, seq_len, page)
    host = O.Cache(pages, H, page, D)
    C.fill_cache(rng, host, table, ctx, k_size=10.0)             # rotated vectors are sqrt(128) times as long
    cache, batch = C.device_cache(torch, host), C.device_batch(torch, table, seq_len, start, T)
    wq, wq_values = weight(torch, hidden, (HQ + 2 * H) * D, 1)
    wo, wo_values = weight(torch, HQ * D, hidden, 2)
    gamma = C.put(torch, (1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32))
    tab = C.rope_table(int(seq_len.max()), D)
    x, h = (rng.standard_normal((T, hidden)).astype(np.float32) for _ in range(2))

    hd = C.put(torch, h)
    q8, s8, hsum = B.add_rmsnorm_quant_i8(C.put(torch, x), gamma, hd)
    y = (B.w8a8_gemv if T <= B.RAD_GEMV_MAX_M else B.w8a8_gemm)(q8, s8, wq)[0]
    qkv = y.view(T, HQ + 2 * H, D)
    q, k, v = qkv.split([HQ, H, H], dim=1)
    q = B.kv4_append(cache, batch, k, v, q, rope=C.put(torch, tab))
    o = B.attn_kv4(cache, batch, q, sm_scale=D ** -0.5)
    oq, os_ = B.quant_act_i8(o.view(T, HQ * D), rotate=False)    # the output is already rotated
    yo = (B.w8a8_gemv if T <= B.RAD_GEMV_MAX_M else B.w8a8_gemm)(oq, os_, wo)[0]
    q2, s2, h2 = B.add_rmsnorm_quant_i8(yo, gamma, hsum)
    torch.cuda.synchronize()

    # each step from what the one before left
    _, n, _ = O.add_rmsnorm(x, h, gamma.cpu().numpy(), 1e-6, "f32", True)
    linear_within_quantisation(y.cpu().numpy(), n, wq_values, s8.cpu().numpy().astype(np.float64))
    yq = y.cpu().numpy().reshape(T, HQ + 2 * H, D)
    for b, m in enumerate(new):
        for i in range(m):
            row, pos = int(start[b]) + i, int(seq_len[b]) - m + i
            q1, k1, v1 = O.append_f32(yq[row:row + 1, :HQ], yq[row:row + 1, HQ:HQ + H], yq[row:row + 1, HQ + H:],
                                      tab[pos:pos + 1], 0, True)
            host.put(int(table[b, pos // page]), pos % page, (k1[0][0], k1[1][0]), (v1[0][0], v1[1][0]))
            assert np.array_equal(q[row].cpu().numpy(), q1[0])
    want, mass, reach = O.attention(q.cpu().numpy(), host, table, seq_len, start, D ** -0.5, True, 0)
    got = o.cpu().numpy()
    assert np.all(np.abs(got - want) <= C.attention_tolerance("f32", want, mass, reach, int(seq_len.max())))
    linear_within_quantisation(yo.cpu().numpy(), got.reshape(T, -1).astype(np.float64), wo_values,
                               os_.cpu().numpy().astype(np.float64))
    assert np.array_equal(h2.cpu().numpy(), x + h + yo.cpu().numpy())
    # against attention with nothing rotated and nothing in 4 bits but what the cache held before: the rotations
    # cancel (q.k and the output projection see them on both sides), so a plain head agrees but for the codes' error
    plain_q = O.turn_f32(yq[:1, :HQ], tab[int(seq_len[0]) - new[0]:int(seq_len[0]) - new[0] + 1], 0)
    assert np.allclose(O.rotate(q.cpu().numpy()[:1]), plain_q, rtol=0, atol=1e-4 * np.abs(plain_q).max())


def test_token_by_token_equals_at_once(torch):
    # one causal call over 40 new rows sees for each row what a call for that row alone, made in its turn, sees
    rng = np.random.default_rng(4)
    n, ctx, H, G, D, page = 40, 55, 2, 3, 128, 32
    table = np.array([[2, 0, 3, 1]], np.int32)
    host = O.Cache(4, H, page, D, rng)
    C.fill_cache(rng, host, table, [ctx], k_size=10.0)
    x = C.put(torch, 3 * rng.standard_normal((n, H * G + 2 * H, D)).astype(np.float32))
    q, k, v = x.split([H * G, H, H], dim=1)
    tab = C.put(torch, C.rope_table(128, D))
    a, b = C.device_cache(torch, host), C.device_cache(torch, host)
    whole = C.device_batch(torch, table, [ctx + n], C.ragged([n]), n)
    qa = B.kv4_append(a, whole, k, v, q, rope=tab)
    oa = B.attn_kv4(a, whole, qa, D ** -0.5).cpu().numpy()
    length = C.put(torch, np.array([ctx], np.int32))
    batch = B.KVBatch(C.put(torch, table), length)               # its length moves on by itself
    rows = []
    for i in range(n):
        length += 1
        qi = B.kv4_append(b, batch, k[i:i + 1], v[i:i + 1], q[i:i + 1], rope=tab)
        rows.append(B.attn_kv4(b, batch, qi, D ** -0.5))
    ob = torch.cat(rows).cpu().numpy()
    for row in range(n):
        host_now = O.Cache(4, H, page, D)
        for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
            getattr(host_now, name)[:] = getattr(b, name).cpu().numpy()
        if row in (0, 17, n - 1):
            want, mass, reach = O.attention(qa[row:row + 1].cpu().numpy(), host_now, table, np.array([ctx + row + 1]),
                                            np.array([0, 1]), D ** -0.5, True, 0)
            tol = C.attention_tolerance("f32", want, mass, reach, ctx + n)
            assert np.all(np.abs(oa[row] - want[0]) <= tol[0]) and np.all(np.abs(ob[row] - want[0]) <= tol[0])


@pytest.mark.parametrize("dtype,n", [("f32", 1), ("bf16", 1), ("bf16", 16), ("f16", 70)])
def test_graph_replays_follow_the_lengths(torch, dtype, n):
    print("graph", dtype, n, flush=True)
    rng = np.random.default_rng(n)
    B_, H, G, D, page, hidden = 3, 2, 5, 128, 64, 1024
    T, cap = B_ * n, 10
    table = rng.permutation(B_ * cap).reshape(B_, cap).astype(np.int32)
    dt = C.torch_dtype(torch, dtype)
    lens = C.put(torch, np.array([n, n + 65, n + 300], np.int32))
    cache = B.KV4Cache.empty(B_ * cap, H, page, D)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        getattr(cache, name).zero_()
    batch = B.KVBatch(C.put(torch, table), lens, None if n == 1 else C.put(torch, C.ragged([n] * B_)), rows=T, max_q=n)
    qkv = torch.randn((T, G * H + 2 * H, D), device="cuda").to(dt)
    q, k, v = qkv.split([G * H, H, H], dim=1)
    x, h, gamma = torch.randn((T, hidden), device="cuda").to(dt), torch.randn((T, hidden), device="cuda").to(dt), torch.ones(hidden, device="cuda")
    tab = C.put(torch, C.rope_table(cap * page, D))
    q_out, o = torch.empty((T, G * H, D), dtype=dt, device="cuda"), torch.empty((T, G * H, D), dtype=dt, device="cuda")
    q8, s8, ho = torch.empty((T, hidden), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(h)
    kr, vr = (torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(max(1, B.attn_kv4_workspace(cache, batch, G * H, dt)), dtype=torch.uint8, device="cuda")
    outs = (q_out, o, q8, s8, ho, kr, vr)

    def step():
        B.add_rmsnorm_quant_i8(x, gamma, h, q=q8, scale=s8, residual_out=ho)
        B.kv4_append(cache, batch, k, v, q, rope=tab, q_out=q_out)
        B.attn_kv4(cache, batch, q_out, 0.05, o=o, workspace=ws)
        B.kv4_read(cache, batch, k=kr, v=vr)

    def bits():
        return [t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32).clone()
                for t in outs]
    step()
    torch.cuda.synchronize()
    state = [getattr(cache, name).clone() for name in ("k_codes", "v_codes", "k_scale", "v_scale")]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(REPLAYS):
        qkv.add_(0.25)                                           # eager work between the replays: new rows ...
        lens.add_(n if r < 2 else 0)                             # ... and longer sequences
        for name, s in zip(("k_codes", "v_codes", "k_scale", "v_scale"), state):
            getattr(cache, name).copy_(s)
        step()
        torch.cuda.synchronize()
        want, after = bits(), [getattr(cache, name).clone() for name in ("k_codes", "v_codes", "k_scale", "v_scale")]
        for name, s in zip(("k_codes", "v_codes", "k_scale", "v_scale"), state):
            getattr(cache, name).copy_(s)
        for t in outs:
            t.fill_(-1 if t.dtype == torch.int8 else float("nan"))
        ws.fill_(255)                                            # NaN in every float
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(bits(), want)):
            assert torch.equal(a, b), "replay %d: output %d differs" % (r, i)
        for name, s in zip(("k_codes", "v_codes", "k_scale", "v_scale"), after):
            assert torch.equal(getattr(cache, name).view(torch.uint8), s.view(torch.uint8)), name
        state = after


def test_two_streams_at_once(torch):
    rng = np.random.default_rng(6)
    H, G, D, page = 2, 5, 128, 64
    jobs = []
    for n, ctx, dtype in ((1, 3000, "f32"), (40, 900, "bf16"), (1, 60, "f16")):
        seq_len = np.array([ctx + n, ctx // 2 + n])
        table, pages = C.page_table(rng, seq_len, page)
        host = O.Cache(pages, H, page, D, rng)
        host.k_scale[:], host.v_scale[:] = np.float16(0.2), np.float16(0.4)
        q = O.to_dtype(rng.standard_normal((2 * n, H * G, D)), dtype)
        start = C.ragged([n, n])
        want, mass, reach = O.attention(q, host, table, seq_len, start, 0.1, True, 0)
        jobs.append((C.device_cache(torch, host), C.device_batch(torch, table, seq_len, start, 2 * n, n), C.put(torch, q, dtype),
                     want, C.attention_tolerance(dtype, want, mass, reach, int(seq_len.max()))))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for (cache, batch, q, _, _), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                outs.append(B.attn_kv4(cache, batch, q, 0.1))
        torch.cuda.synchronize()
        for o, (_, _, _, want, tol) in zip(outs, jobs):
            assert np.all(np.abs(C.host(o) - want) <= tol)


def test_offsets_past_32_bits(torch):
    # 34,000 pages of 128 KiB: codes reach past 2^32 bytes; the sequence lies on the first and the last pages
    rng = np.random.default_rng(7)
    pages, H, page, D, G = 34000, 8, 256, 128, 1
    cache = B.KV4Cache.empty(pages, H, page, D)
    assert cache.k_codes.numel() > 2 ** 32
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    small = np.array([[2, 0, 1]], np.int32)
    n = 2 * page + 77
    x = C.put(torch, rng.standard_normal((n, H * G + 2 * H, D)).astype(np.float32))
    q, k, v = x.split([H * G, H, H], dim=1)
    ref = B.KV4Cache.empty(3, H, page, D)
    outs = []
    for c, t in ((cache, table), (ref, small)):
        batch = C.device_batch(torch, t, [n], C.ragged([n]), n)
        qo = B.kv4_append(c, batch, k, v, q)
        one = B.KVBatch(C.put(torch, t), C.put(torch, np.array([n], np.int32)))
        outs.append((qo, B.attn_kv4(c, batch, qo, 0.1), B.attn_kv4(c, one, qo[-1:].contiguous(), 0.1), *B.kv4_read(c, batch)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_many_sequences(torch):
    # more than the 64 that a wave looks at at once, and more than the 512 whose contexts are cut
    rng = np.random.default_rng(8)
    H, G, D, page = 1, 3, 64, 32
    for nseq in (70, 600):
        new = rng.integers(0, 4, nseq)
        new[5] = 3
        ctx = rng.integers(0, 50, nseq)
        seq_len, start = new + ctx, C.ragged(new)
        table, pages = C.page_table(rng, seq_len, page)
        host = O.Cache(pages, H, page, D, rng)
        host.k_scale[:], host.v_scale[:] = np.float16(0.2), np.float16(0.4)
        T = int(start[-1])
        q = rng.standard_normal((T, H * G, D)).astype(np.float32)
        o = B.attn_kv4(C.device_cache(torch, host), C.device_batch(torch, table, seq_len, start, T, 3), C.put(torch, q), 0.1)
        want, mass, reach = O.attention(q, host, table, seq_len, start, 0.1, True, 0)
        assert np.all(np.abs(C.host(o) - want) <= C.attention_tolerance("f32", want, mass, reach, 60))
        o2 = B.attn_kv4(C.device_cache(torch, host), C.device_batch(torch, table, seq_len, start, T), C.put(torch, q), 0.1)
        assert np.all(np.abs(C.host(o2) - want) <= C.attention_tolerance("f32", want, mass, reach, 60))


@pytest.mark.parametrize("inside", [True, False])
def test_graph_replays_follow_the_block_table(torch, inside):
    # page ids are read anew by every replay, written by the graph itself just before or by work between replays
    rng = np.random.default_rng(21)
    H, G, D, page, B_, width = 2, 4, 128, 32, 3, 40
    host = O.Cache(2 * B_ * width, H, page, D, rng)
    C.fill_cache(rng, host, np.arange(2 * B_ * width, dtype=np.int32)[None], [2 * B_ * width * page])
    cache = C.device_cache(torch, host)
    seq_len = np.array([1000, 1270, 33])
    tables = [rng.permutation(2 * B_ * width)[:B_ * width].reshape(B_, width).astype(np.int32) for _ in range(4)]
    dev = [C.put(torch, t) for t in tables]
    batch = C.device_batch(torch, tables[0], seq_len, None, B_)
    q = O.to_dtype(rng.standard_normal((B_, H * G, D)), "bf16")
    qd, src, o = C.put(torch, q, "bf16"), dev[0].clone(), torch.empty((B_, H * G, D), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.attn_kv4(cache, batch, qd, D ** -0.5, o=o)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            if inside:
                batch.block_table.copy_(src)
            B.attn_kv4(cache, batch, qd, D ** -0.5, o=o)
        for k in (1, 2, 3, 0, 2):
            (src if inside else batch.block_table).copy_(dev[k])
            o.fill_(9.0)
            g.replay()
            s.synchronize()
            want, mass, reach = O.attention(q, host, tables[k], seq_len, C.ragged([1] * B_), D ** -0.5, True, 0)
            tol = C.attention_tolerance("bf16", want, mass, reach, 1270)
            assert np.all(np.abs(C.host(o) - want) <= tol), k


@pytest.mark.parametrize("nseq,most,starts,H,G,D,dtype", [
    (513, 40, True, 2, 3, 64, "bf16"), (700, 40, True, 1, 5, 128, "f32"), (600, 9, True, 2, 7, 256, "f16"),
    (520, 1, False, 1, 40, 64, "f16"), (700, 1, False, 2, 4, 128, "bf16"), (5000, 3, True, 1, 2, 64, "f32"),
    (70000, 2, True, 1, 20, 64, "bf16"), (70000, 1, False, 1, 33, 64, "f32"), (70000, 1, True, 1, 1, 64, "f32")])
def test_more_sequences_than_are_looked_at_by_every_workgroup(torch, nseq, most, starts, H, G, D, dtype):
    # every row written, and a sample of the sequences against the oracle: the first and last, empty ones, the longest
    print("sequences", nseq, most, starts, H, G, D, dtype, flush=True)
    rng = np.random.default_rng(nseq + G)
    page, pool = 32, 50
    new = rng.integers(0, most + 1, nseq) if starts else np.ones(nseq, int)
    if starts:
        new[[0, 7, nseq - 1]], new[[8, 9, nseq - 2]] = most, 0
    seq_len = np.maximum(new + rng.integers(-1, 60, nseq), 0)
    table = rng.integers(-1, pool, (nseq, 4)).astype(np.int32)         # shared pages, some absent
    host = O.Cache(pool, H, page, D, rng)
    host.k_scale[:], host.v_scale[:] = np.float16(0.2), np.float16(0.4)
    start = C.ragged(new)
    T = int(start[-1]) + (5 if starts else 0)
    q = O.to_dtype(rng.standard_normal((T, H * G, D)), dtype)
    o = torch.full(q.shape, float("nan"), dtype=C.torch_dtype(torch, dtype), device="cuda")
    batch = C.device_batch(torch, table, seq_len, start if starts else None, T, most)
    B.attn_kv4(C.device_cache(torch, host), batch, C.put(torch, q, dtype), 0.1, o=o)
    got = C.host(o)
    assert np.isnan(got[start[-1]:]).all() and not np.isnan(got[:start[-1]]).any()
    some = np.unique(np.concatenate([np.arange(12), np.arange(nseq - 70, nseq), rng.integers(0, nseq, 60)]))
    rows = np.concatenate([np.arange(start[b], start[b + 1]) for b in some])
    want, mass, reach = O.attention(q[rows], host, table[some], seq_len[some], C.ragged(new[some]), 0.1, True, 0)
    assert np.all(np.abs(got[rows] - want) <= C.attention_tolerance(dtype, want, mass, reach, 100))


@pytest.mark.parametrize("dtype,n,G,D", [("f32", 1, 5, 128), ("bf16", 16, 5, 128), ("f16", 7, 8, 64), ("bf16", 9, 4, 256)])
def test_graph_replays_of_cut_contexts(torch, dtype, n, G, D):
    # two captured calls with a workspace each; between replays lengths move so that the cut into parts is another,
    # down to sequences of a few tokens, and the workspaces hold NaN
    print("graph cut", dtype, n, G, D, flush=True)
    rng = np.random.default_rng(n + D)
    B_, H, page, width = 3, 2, 64, 140
    host = O.Cache(B_ * width, H, page, D, rng)
    host.k_scale[:] = 0.3 * np.exp(rng.uniform(-0.5, 0.5, host.k_scale.shape))
    host.v_scale[:] = 0.4 * np.exp(rng.uniform(-1, 1, host.v_scale.shape))
    cache, dt = C.device_cache(torch, host), C.torch_dtype(torch, dtype)
    table, start = rng.permutation(B_ * width).reshape(B_, width).astype(np.int32), C.ragged([n] * B_)
    lens = torch.zeros(B_, dtype=torch.int32, device="cuda")
    batch = B.KVBatch(C.put(torch, table), lens, C.put(torch, start), rows=B_ * n, max_q=n)
    q = [O.to_dtype(rng.standard_normal((B_ * n, H * G, D)), dtype) for _ in range(2)]
    qd, o = [C.put(torch, x, dtype) for x in q], [torch.empty((B_ * n, H * G, D), dtype=dt, device="cuda") for _ in range(2)]
    size = B.attn_kv4_workspace(cache, batch, H * G, dt)
    assert size > 0
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def call(i):
        B.attn_kv4(cache, batch, qd[i], 0.1, window=(0, 3000)[i], o=o[i], workspace=ws[i])
    graphs = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for seq_len in ([8960, 4000, 77], [n, 5, 6000], [0, 8960, 8960], [300, 200, 100], [5000, 8000, 2 * n]):
        lens.copy_(torch.tensor(seq_len, dtype=torch.int32))
        for i in range(2):
            call(i)
        torch.cuda.synchronize()
        eager = [x.clone() for x in o]
        for i in range(2):
            o[i].fill_(float("nan"))
            ws[i].fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(o[i].view(torch.uint8), eager[i].view(torch.uint8)), (seq_len, i)
            want, mass, reach = O.attention(q[i], host, table, np.array(seq_len), start, 0.1, True, (0, 3000)[i])
            assert np.all(np.abs(C.host(o[i]) - want) <= C.attention_tolerance(dtype, want, mass, reach, 8960)), (seq_len, i)
