"""The calls between a layer's linears refuse bad arguments on the host, before any HIP call (every call here fails
its checks or is empty).  Fake, never dereferenced addresses stand in for device pointers."""
import ctypes
import os

import pytest

from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="librad.so not built")

P = [0x7F0000000000 + i * 0x10000000000 for i in range(16)]     # aligned, far apart
F32, BF16, F16 = B.RAD_DT_F32, B.RAD_DT_BF16, B.RAD_DT_F16


def test_dtype_constants_match_header():
    h = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "rad.h")).read()
    for name in ("RAD_DT_F32", "RAD_DT_BF16", "RAD_DT_F16"):
        assert "%s = %d" % (name, getattr(B, name)) in h


def norm(x=P[0], r=P[1], ro=P[1], g=P[2], eps=1e-6, q=P[3], s=P[4], M=4, K=256, dt=F32, rot=1):
    return B.lib().rad_add_rmsnorm_quant_i8(x, r, ro, g, eps, q, s, M, K, dt, rot, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), B.RAD_E_FMT), (dict(dt=-1), B.RAD_E_FMT),
    (dict(K=200), B.RAD_E_SHAPE), (dict(K=0), B.RAD_E_SHAPE), (dict(M=-1), B.RAD_E_SHAPE),
    (dict(K=B.RAD_QUANT_MAX_K + 128), B.RAD_E_RANGE), (dict(M=1 << 31), B.RAD_E_RANGE), (dict(rot=2), B.RAD_E_RANGE),
    (dict(eps=-1e-6), B.RAD_E_RANGE), (dict(eps=float("nan")), B.RAD_E_RANGE), (dict(eps=float("inf")), B.RAD_E_RANGE),
    (dict(r=None), B.RAD_E_NULL), (dict(ro=None), B.RAD_E_NULL), (dict(x=None), B.RAD_E_NULL),
    (dict(g=None), B.RAD_E_NULL), (dict(q=None), B.RAD_E_NULL), (dict(s=None), B.RAD_E_NULL),
    (dict(x=P[0] + 8), B.RAD_E_ALIGN), (dict(r=P[1] + 8, ro=P[5]), B.RAD_E_ALIGN), (dict(ro=P[5] + 4), B.RAD_E_ALIGN),
    (dict(g=P[2] + 4), B.RAD_E_ALIGN), (dict(q=P[3] + 4), B.RAD_E_ALIGN), (dict(s=P[4] + 2), B.RAD_E_ALIGN),
    (dict(q=P[0] + 1024), B.RAD_E_ALIAS), (dict(s=P[3] + 512), B.RAD_E_ALIAS), (dict(ro=P[1] + 2048), B.RAD_E_ALIAS),
    (dict(ro=P[0]), B.RAD_E_ALIAS), (dict(x=P[1]), B.RAD_E_ALIAS), (dict(g=P[1] + 256), B.RAD_E_ALIAS),
    (dict(q=P[1] + 4 * 256 * 4 - 16), B.RAD_E_ALIAS),
    (dict(M=0, x=None, r=None, ro=None, g=None, q=None, s=None), B.RAD_OK),
])
def test_norm_refusals(kw, rc):
    assert norm(**kw) == rc


def test_more_than_a_launch_holds():
    assert norm(M=(1 << 24) - 1, r=None, ro=None, x=None) == B.RAD_E_NULL          # the size itself is taken
    assert norm(M=1 << 24, r=None, ro=None) == B.RAD_E_RANGE
    big = dict(heads=1024, D=256)
    assert read(c=big, b=dict(rows=1 << 17)) == B.RAD_E_RANGE
    assert read(c=big, b=dict(rows=(1 << 17) - 1), k=None) == B.RAD_E_NULL


def cache(k=P[0], ks=P[1], v=P[2], vs=P[3], pages=10, heads=2, page=64, D=128):
    return B.KV4CacheDesc(k, ks, v, vs, pages, heads, page, D)


def batch(table=P[4], n=P[5], start=P[6], seqs=3, max_pages=4, rows=7, max_q=7):
    return B.KVBatchDesc(table, n, start, seqs, max_pages, rows, max_q)


CACHE_REFUSALS = [
    (dict(D=96), B.RAD_E_SHAPE), (dict(D=0), B.RAD_E_SHAPE), (dict(page=16), B.RAD_E_SHAPE),
    (dict(page=48), B.RAD_E_SHAPE), (dict(page=512), B.RAD_E_SHAPE), (dict(pages=0), B.RAD_E_SHAPE),
    (dict(heads=0), B.RAD_E_SHAPE), (dict(heads=1025), B.RAD_E_RANGE), (dict(pages=1 << 31), B.RAD_E_RANGE),
    (dict(k=None), B.RAD_E_NULL), (dict(ks=None), B.RAD_E_NULL), (dict(v=None), B.RAD_E_NULL),
    (dict(vs=None), B.RAD_E_NULL), (dict(k=P[0] + 8), B.RAD_E_ALIGN), (dict(ks=P[1] + 2), B.RAD_E_ALIGN),
    (dict(v=P[2] + 4), B.RAD_E_ALIGN), (dict(vs=P[3] + 8), B.RAD_E_ALIGN),
]
BATCH_REFUSALS = [
    (dict(seqs=-1), B.RAD_E_SHAPE), (dict(rows=-1), B.RAD_E_SHAPE), (dict(max_pages=-1), B.RAD_E_SHAPE),
    (dict(max_q=-1), B.RAD_E_SHAPE), (dict(start=None), B.RAD_E_SHAPE),       # rows != B without q_start
    (dict(seqs=1 << 24), B.RAD_E_RANGE), (dict(rows=1 << 24), B.RAD_E_RANGE),
    (dict(max_pages=1 << 24), B.RAD_E_RANGE), (dict(max_pages=1 << 40), B.RAD_E_RANGE),
    (dict(table=None), B.RAD_E_NULL), (dict(n=None), B.RAD_E_NULL),
    (dict(table=P[4] + 2), B.RAD_E_ALIGN), (dict(n=P[5] + 1), B.RAD_E_ALIGN), (dict(start=P[6] + 2), B.RAD_E_ALIGN),
]


def append(c={}, b={}, k=P[7], ldk=256, v=P[8], ldv=256, q=P[9], ldq=512, q_heads=4, qo=P[10], rope=None, rot=1,
           dt=BF16):
    return B.lib().rad_kv4_append(cache(**c), batch(**b), k, ldk, v, ldv, q, ldq, q_heads, qo,
                                  None if rope is None else B.RopeDesc(*rope), rot, dt, None)


def read(c={}, b={}, k=P[7], v=P[8]):
    return B.lib().rad_kv4_read(cache(**c), batch(**b), k, v, None)


def attn(c={}, b={}, q=P[7], q_heads=4, scale=0.1, causal=1, window=0, o=P[8], ws=P[9], ws_bytes=1 << 40, dt=BF16):
    return B.lib().rad_attn_kv4(cache(**c), batch(**b), q, q_heads, scale, causal, window, o, ws, ws_bytes, dt, None)


@pytest.mark.parametrize("call", [append, read, attn])
@pytest.mark.parametrize("kw,rc", CACHE_REFUSALS)
def test_cache_refusals(call, kw, rc):
    assert call(c=kw) == rc


@pytest.mark.parametrize("call", [append, read, attn])
@pytest.mark.parametrize("kw,rc", BATCH_REFUSALS)
def test_batch_refusals(call, kw, rc):
    assert call(b=kw) == rc


@pytest.mark.parametrize("call", [append, read, attn])
@pytest.mark.parametrize("kw", [dict(rows=0), dict(seqs=0)])
def test_empty_batches_enqueue_nothing(call, kw):
    assert call(b=dict(kw, table=None, n=None)) == B.RAD_OK


def test_an_empty_append_needs_no_arrays():
    # empty tensors have no address
    for kw in (dict(rows=0), dict(seqs=0)):
        assert append(b=kw, k=None, v=None, q=None, qo=None) == B.RAD_OK
        assert append(b=kw, q=None) == B.RAD_OK


@pytest.mark.parametrize("call", ["append", "read", "attn", "workspace"])
def test_missing_descriptors(call):
    L, n = B.lib(), ctypes.c_int64(0)
    for c, b in ((None, batch()), (cache(), None)):
        rc = {"append": lambda: L.rad_kv4_append(c, b, P[7], 256, P[8], 256, None, 0, 0, None, None, 0, BF16, None),
              "read": lambda: L.rad_kv4_read(c, b, P[7], P[8], None),
              "attn": lambda: L.rad_attn_kv4(c, b, P[7], 4, 0.1, 1, 0, P[8], P[9], 1 << 40, BF16, None),
              "workspace": lambda: L.rad_attn_kv4_workspace(c, b, 4, BF16, ctypes.byref(n))}[call]()
        assert rc == B.RAD_E_NULL


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=5), B.RAD_E_FMT), (dict(rot=2), B.RAD_E_RANGE),
    (dict(c=dict(D=64), rot=1), B.RAD_E_SHAPE),                               # the rotation needs 128s
    (dict(ldk=255), B.RAD_E_SHAPE), (dict(ldv=0), B.RAD_E_SHAPE), (dict(ldq=511), B.RAD_E_SHAPE),
    (dict(q_heads=-1), B.RAD_E_SHAPE), (dict(q_heads=16385, ldq=1 << 22), B.RAD_E_RANGE),
    (dict(ldk=1 << 31), B.RAD_E_RANGE),
    (dict(rope=(P[11], 100, 12, 0)), B.RAD_E_SHAPE), (dict(rope=(P[11], 100, 136, 0)), B.RAD_E_SHAPE),
    (dict(rope=(P[11], 100, 0, 0)), B.RAD_E_SHAPE), (dict(rope=(P[11], -1, 64, 0)), B.RAD_E_SHAPE),
    (dict(rope=(P[11], 100, 64, 2)), B.RAD_E_RANGE), (dict(rope=(P[11], 1 << 31, 64, 0)), B.RAD_E_RANGE),
    (dict(rope=(None, 100, 64, 0)), B.RAD_E_NULL), (dict(rope=(P[11] + 4, 100, 64, 0)), B.RAD_E_ALIGN),
    (dict(q=None), B.RAD_E_NULL), (dict(qo=None), B.RAD_E_NULL), (dict(q=None, q_heads=0), B.RAD_E_NULL),
    (dict(k=None), B.RAD_E_NULL), (dict(v=None), B.RAD_E_NULL),
    (dict(k=P[7] + 8), B.RAD_E_ALIGN), (dict(v=P[8] + 2), B.RAD_E_ALIGN), (dict(q=P[9] + 4), B.RAD_E_ALIGN),
    (dict(qo=P[10] + 8), B.RAD_E_ALIGN), (dict(ldk=260), B.RAD_E_ALIGN), (dict(ldq=518, dt=F32), B.RAD_E_ALIGN),
    (dict(qo=P[9] + 1024), B.RAD_E_ALIAS), (dict(qo=P[7]), B.RAD_E_ALIAS), (dict(k=P[0] + 4096), B.RAD_E_ALIAS),
    (dict(v=P[3]), B.RAD_E_ALIAS), (dict(qo=P[2]), B.RAD_E_ALIAS), (dict(qo=P[5]), B.RAD_E_ALIAS),
    (dict(b=dict(n=P[1] + 64)), B.RAD_E_ALIAS), (dict(c=dict(ks=P[0] + 1024)), B.RAD_E_ALIAS),
    (dict(rope=(P[2], 100, 64, 0)), B.RAD_E_ALIAS), (dict(rope=(P[10], 100, 64, 0)), B.RAD_E_ALIAS),
])
def test_append_refusals(kw, rc):
    assert append(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), B.RAD_E_NULL), (dict(v=None), B.RAD_E_NULL), (dict(k=P[7] + 8), B.RAD_E_ALIGN),
    (dict(v=P[8] + 4), B.RAD_E_ALIGN), (dict(v=P[7] + 256), B.RAD_E_ALIAS), (dict(k=P[2]), B.RAD_E_ALIAS),
    (dict(v=P[4]), B.RAD_E_ALIAS),
])
def test_read_refusals(kw, rc):
    assert read(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), B.RAD_E_FMT), (dict(q_heads=0), B.RAD_E_SHAPE), (dict(q_heads=5), B.RAD_E_SHAPE),
    (dict(q_heads=1 << 15), B.RAD_E_RANGE), (dict(b=dict(rows=(1 << 24) - 1), q_heads=1024), B.RAD_E_RANGE),
    (dict(scale=0.0), B.RAD_E_RANGE), (dict(scale=-1.0), B.RAD_E_RANGE), (dict(scale=float("nan")), B.RAD_E_RANGE),
    (dict(scale=float("inf")), B.RAD_E_RANGE), (dict(scale=2.0 ** 126.5), B.RAD_E_RANGE), (dict(causal=2), B.RAD_E_RANGE), (dict(window=-1), B.RAD_E_SHAPE),
    (dict(q=None), B.RAD_E_NULL), (dict(o=None), B.RAD_E_NULL), (dict(q=P[7] + 8), B.RAD_E_ALIGN),
    (dict(o=P[8] + 4), B.RAD_E_ALIGN), (dict(ws=P[9] + 8), B.RAD_E_ALIGN), (dict(o=P[7] + 64), B.RAD_E_ALIAS),
    (dict(o=P[0] + 64), B.RAD_E_ALIAS), (dict(o=P[6]), B.RAD_E_ALIAS),
])
def test_attention_refusals(kw, rc):
    assert attn(**kw) == rc


def test_binding_refuses_host_tensors():
    import torch
    x, g = torch.zeros(2, 256), torch.ones(256)
    with pytest.raises(TypeError, match="GPU tensor"):
        B.add_rmsnorm_quant_i8(x, g)
    u8 = torch.zeros(1, 1, 32, 64, dtype=torch.uint8)
    with pytest.raises(TypeError, match="GPU tensor"):
        B.KV4Cache(u8, torch.zeros(1, 1, 32).half(), u8.view(1, 1, 4, 128, 4), torch.zeros(1, 1, 32).half())
    with pytest.raises(TypeError, match="GPU tensor"):
        B.KVBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("max_pages", [4, 64, 4096])
def test_attention_of_no_rows_a_sequence_is_done_at_once(max_pages):
    # max_q 0: every row is past it and stays as it was, whatever the table's width
    n, kw = ctypes.c_int64(-1), dict(max_q=0, max_pages=max_pages)
    assert B.lib().rad_attn_kv4_workspace(cache(), batch(**kw), 4, BF16, ctypes.byref(n)) == B.RAD_OK and n.value == 0
    assert attn(b=kw, ws=None, ws_bytes=0) == B.RAD_OK
    assert attn(b=kw, q_heads=5) == B.RAD_E_SHAPE             # its sizes are still looked at


def test_norm_of_more_threads_than_a_launch_holds():
    # wide tokens take more threads each: up to 1024, 64 for every 1024 values
    one = dict(r=None, ro=None)
    for K, most in ((2048, (1 << 24) - 1), (4096, (1 << 24) - 1), (5120, (1 << 32) // 320), (8192, (1 << 23) - 1),
                    (8320, (1 << 32) // 576), (65536, (1 << 22) - 1)):
        assert norm(M=most, K=K, x=None, **one) == B.RAD_E_NULL, K       # the size itself is taken
        assert norm(M=most + 1, K=K, x=None, **one) == B.RAD_E_RANGE, K


def test_read_back_of_more_threads_than_a_launch_holds():
    # 2048 values a workgroup of 256 threads: one value short of 2^35 still rounds up to 2^24 workgroups
    assert read(c=dict(heads=233, D=64), b=dict(rows=2304167)) == B.RAD_E_RANGE      # 2^35 - 64 values
    assert read(c=dict(heads=1, D=64), b=dict(rows=(1 << 22) - 1), k=None) == B.RAD_E_NULL


def test_attention_of_more_workgroups_than_a_launch_holds():
    # 256 threads a tile of 32 (row, head) pairs of a KV head, 16 for heads of 256, and a tile more a sequence
    n, one = ctypes.c_int64(0), dict(seqs=1, max_pages=1)

    def both(c, b, q_heads, rc):
        assert attn(c=c, b=b, q_heads=q_heads, q=None, ws_bytes=1 << 60) == rc
        assert B.lib().rad_attn_kv4_workspace(cache(**c), batch(**b), q_heads, BF16,
                                              ctypes.byref(n)) == (B.RAD_OK if rc == B.RAD_E_NULL else rc)
    many = dict(seqs=1024, max_pages=1)
    both(dict(heads=1, D=64), dict(many, rows=32767, max_q=32767), 16384, B.RAD_E_RANGE)      # 2^24 + 512
    both(dict(heads=1, D=64), dict(many, rows=32765, max_q=32765), 16384, B.RAD_E_NULL)       # 2^24 - 512
    both(dict(heads=1, D=64), dict(one, rows=32767, max_q=32767), 16384, B.RAD_E_NULL)        # 2^24 - 511
    both(dict(heads=1, D=256), dict(many, rows=16383, max_q=16383), 16384, B.RAD_E_RANGE)     # 2^24
    both(dict(heads=1, D=256), dict(one, rows=32767, max_q=32767), 16384, B.RAD_E_RANGE)      # nearly 2^25
    both(dict(heads=1, D=256), dict(many, rows=16382, max_q=16382), 16384, B.RAD_E_NULL)
    both(dict(heads=2, D=256), dict(many, rows=32767, max_q=32767), 16384, B.RAD_E_RANGE)
    both(dict(heads=4, D=256), dict(many, rows=32767, max_q=32767), 16384, B.RAD_E_NULL)
