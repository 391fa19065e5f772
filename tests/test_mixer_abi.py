"""The token mixers' calls refuse bad arguments on the host, before any HIP call (every call here fails its checks or is
empty).  Fake, never dereferenced addresses stand in for device pointers."""
import ctypes
import os

import pytest

from rotated_w8a8_int8_amd import binding as B
from test_layer_abi import BATCH_REFUSALS, BF16, CACHE_REFUSALS, F32, P, batch, cache

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="librad.so not built")

NAN, INF = float("nan"), float("inf")


def append_at(c={}, b={}, k=P[7], v=P[8], q=P[9], qo=P[10], rope=(P[11], 100, 64, 0), pos=P[12], dt=BF16):
    return B.lib().rad_kv4_append_at(cache(**c), batch(**b), k, 256, v, 256, q, 512, 4, qo, B.RopeDesc(*rope), pos, 1,
                                     dt, None)


def tree(c={}, b={}, q=P[7], q_heads=4, scale=0.1, mask=P[10], words=1, window=0, o=P[8], ws=P[9], ws_bytes=1 << 40, dt=BF16):
    return B.lib().rad_attn_kv4_tree(cache(**c), batch(**b), q, q_heads, scale, mask, words, window, o, ws, ws_bytes, dt, None)


def weights(c={}, b={}, q=P[7], q_heads=4, scale=0.1, causal=1, window=0, o=P[8], w=P[10], ldw=256, observe=0, factor=1.0,
            ws=P[9], ws_bytes=1 << 40, dt=BF16):
    return B.lib().rad_attn_kv4_weights(cache(**c), batch(**b), q, q_heads, scale, causal, window, o, w, ldw, observe, factor,
                                        ws, ws_bytes, dt, None)


def select(w=P[0], ldw=512, n=P[1], seqs=3, heads=2, tokens=500, budget=64, first=4, recent=8, kept=P[2], count=P[3],
           kw=P[4], ldk=64, ws=P[5], ws_bytes=1 << 40):
    return B.lib().rad_kv4_select(w, ldw, n, seqs, heads, tokens, budget, first, recent, kept, count, kw, ldk, ws, ws_bytes, None)


def other(**kw):
    return cache(**dict(dict(k=P[11], ks=P[12], v=P[13], vs=P[14]), **kw))


def move(c={}, b={}, src=P[7], lists=2, entries=64, count=P[8], to="none", table=P[9], pages=3, start=P[10]):
    to = None if to == "none" else other(**to)
    return B.lib().rad_kv4_move(cache(**c), batch(**b), src, lists, entries, count, to, table, pages, start, None)


def linear(q=P[0], k=P[1], v=P[2], ldq=256, ldk=256, ldv=512, g=P[3], start=P[4], seqs=3, rows=7, max_q=7, qk=2, heads=4,
           D=128, dt=BF16, s=P[5], so=P[6], scale=1.0, o=P[7], ws=P[8], ws_bytes=1 << 40):
    d = B.LinearDesc(q, k, v, ldq, ldk, ldv, g, start, seqs, rows, max_q, qk, heads, D, dt)
    return B.lib().rad_linear_attn(d, s, so, scale, o, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [append_at, tree, weights, move])
@pytest.mark.parametrize("kw,rc", CACHE_REFUSALS)
def test_cache_refusals(call, kw, rc):
    assert call(c=kw, **(dict(lists=1) if call is move else {})) == rc


@pytest.mark.parametrize("call", [append_at, tree, weights])
@pytest.mark.parametrize("kw,rc", BATCH_REFUSALS)
def test_batch_refusals(call, kw, rc):
    # a row of weights is long enough for no such batch
    if call is weights and kw.get("max_pages", 0) > 4:
        kw = dict(kw)
        assert call(b=kw, ldw=1 << 20) in (rc, B.RAD_E_SHAPE)
        return
    assert call(b=kw) == rc


@pytest.mark.parametrize("call", [append_at, tree, weights])
@pytest.mark.parametrize("kw", [dict(rows=0), dict(seqs=0)])
def test_empty_batches_enqueue_nothing(call, kw):
    assert call(b=dict(kw, table=None, n=None)) == B.RAD_OK


@pytest.mark.parametrize("kw,rc", [
    (dict(pos=P[12] + 2), B.RAD_E_ALIGN), (dict(pos=P[0] + 4096), B.RAD_E_ALIAS), (dict(pos=P[10]), B.RAD_E_ALIAS),
    (dict(dt=5), B.RAD_E_FMT), (dict(rope=(P[11], 100, 12, 0)), B.RAD_E_SHAPE), (dict(k=None), B.RAD_E_NULL),
    (dict(qo=P[9] + 1024), B.RAD_E_ALIAS),
])
def test_append_refusals(kw, rc):
    assert append_at(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), B.RAD_E_FMT), (dict(q_heads=0), B.RAD_E_SHAPE), (dict(q_heads=5), B.RAD_E_SHAPE),
    (dict(q_heads=1 << 15), B.RAD_E_RANGE), (dict(scale=0.0), B.RAD_E_RANGE), (dict(scale=NAN), B.RAD_E_RANGE),
    (dict(scale=INF), B.RAD_E_RANGE), (dict(window=-1), B.RAD_E_SHAPE), (dict(words=0), B.RAD_E_RANGE),
    (dict(words=-1), B.RAD_E_RANGE), (dict(words=B.RAD_TREE_MAX_WORDS + 1), B.RAD_E_RANGE),
    (dict(q=None), B.RAD_E_NULL), (dict(o=None), B.RAD_E_NULL), (dict(mask=None), B.RAD_E_NULL),
    (dict(mask=P[10] + 4), B.RAD_E_ALIGN), (dict(o=P[8] + 4), B.RAD_E_ALIGN), (dict(ws=P[9] + 8), B.RAD_E_ALIGN),
    (dict(o=P[7] + 64), B.RAD_E_ALIAS), (dict(o=P[10]), B.RAD_E_ALIAS), (dict(o=P[0] + 64), B.RAD_E_ALIAS),
    (dict(b=dict(max_pages=64), ws=P[10]), B.RAD_E_ALIAS), (dict(b=dict(max_pages=64), ws_bytes=64), B.RAD_E_RANGE),
    (dict(b=dict(max_pages=64), ws=None), B.RAD_E_NULL),
])
def test_tree_refusals(kw, rc):
    assert tree(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), B.RAD_E_FMT), (dict(q_heads=5), B.RAD_E_SHAPE), (dict(causal=2), B.RAD_E_RANGE),
    (dict(window=-1), B.RAD_E_SHAPE), (dict(scale=-1.0), B.RAD_E_RANGE), (dict(ldw=252), B.RAD_E_SHAPE),
    (dict(ldw=258), B.RAD_E_SHAPE), (dict(ldw=1 << 31), B.RAD_E_RANGE), (dict(observe=-1), B.RAD_E_SHAPE),
    (dict(factor=-0.5), B.RAD_E_RANGE), (dict(factor=NAN), B.RAD_E_RANGE), (dict(factor=INF), B.RAD_E_RANGE),
    (dict(w=None), B.RAD_E_NULL), (dict(o=None), B.RAD_E_NULL), (dict(ws=None), B.RAD_E_NULL),
    (dict(ws_bytes=64), B.RAD_E_RANGE), (dict(w=P[10] + 8), B.RAD_E_ALIGN), (dict(w=P[7]), B.RAD_E_ALIAS),
    (dict(w=P[8]), B.RAD_E_ALIAS), (dict(w=P[9]), B.RAD_E_ALIAS), (dict(w=P[2] + 64), B.RAD_E_ALIAS),
    (dict(w=P[5]), B.RAD_E_ALIAS),
])
def test_weights_refusals(kw, rc):
    assert weights(**kw) == rc


def test_workspaces():
    L, n, m = B.lib(), ctypes.c_int64(0), ctypes.c_int64(0)
    for c, b in ((None, batch()), (cache(), None)):
        assert L.rad_attn_kv4_weights_workspace(c, b, 4, BF16, ctypes.byref(n)) == B.RAD_E_NULL
        assert L.rad_kv4_move(c, b, P[7], 1, 4, P[8], None, None, 0, None, None) == B.RAD_E_NULL
    assert L.rad_attn_kv4_weights_workspace(cache(), batch(), 4, BF16, None) == B.RAD_E_NULL
    assert L.rad_attn_kv4_workspace(cache(), batch(), 4, BF16, ctypes.byref(n)) == B.RAD_OK
    assert L.rad_attn_kv4_weights_workspace(cache(), batch(), 4, BF16, ctypes.byref(m)) == B.RAD_OK
    assert m.value >= n.value + 7 * 4 * 8                    # a row's statistics: two f32 a head
    assert L.rad_kv4_select_workspace(3, 2, 500, None) == B.RAD_E_NULL
    assert L.rad_kv4_select_workspace(0, 2, 500, ctypes.byref(n)) == B.RAD_OK and n.value == 0
    assert L.rad_kv4_select_workspace(-1, 2, 500, ctypes.byref(n)) == B.RAD_E_SHAPE
    assert L.rad_linear_attn_workspace(None, ctypes.byref(n)) == B.RAD_E_NULL
    assert L.rad_linear_attn(None, None, None, 1.0, None, None, 0, None) == B.RAD_E_NULL


@pytest.mark.parametrize("kw,rc", [
    (dict(seqs=-1), B.RAD_E_SHAPE), (dict(heads=-1), B.RAD_E_SHAPE), (dict(tokens=-1), B.RAD_E_SHAPE),
    (dict(budget=0), B.RAD_E_SHAPE), (dict(first=-1), B.RAD_E_SHAPE), (dict(recent=-1), B.RAD_E_SHAPE),
    (dict(ldw=499), B.RAD_E_SHAPE), (dict(ldw=502), B.RAD_E_SHAPE), (dict(ldk=63), B.RAD_E_SHAPE),
    (dict(seqs=1 << 22), B.RAD_E_RANGE), (dict(heads=1025), B.RAD_E_RANGE), (dict(seqs=1 << 12, heads=1024), B.RAD_E_RANGE),
    (dict(tokens=1 << 30, ldw=1 << 30), B.RAD_E_RANGE), (dict(budget=1 << 30, ldk=1 << 30), B.RAD_E_RANGE),
    (dict(first=60), B.RAD_E_RANGE), (dict(first=65, recent=0), B.RAD_E_RANGE), (dict(ldw=1 << 31), B.RAD_E_RANGE),
    (dict(w=None), B.RAD_E_NULL), (dict(n=None), B.RAD_E_NULL), (dict(kept=None), B.RAD_E_NULL), (dict(count=None), B.RAD_E_NULL),
    (dict(w=P[0] + 4), B.RAD_E_ALIGN), (dict(n=P[1] + 2), B.RAD_E_ALIGN), (dict(kept=P[2] + 1), B.RAD_E_ALIGN),
    (dict(count=P[3] + 2), B.RAD_E_ALIGN), (dict(kw=P[4] + 2), B.RAD_E_ALIGN),
    (dict(kept=P[0]), B.RAD_E_ALIAS), (dict(count=P[2] + 64), B.RAD_E_ALIAS), (dict(kw=P[0] + 1024), B.RAD_E_ALIAS),
    (dict(count=P[1]), B.RAD_E_ALIAS), (dict(seqs=0, w=None, n=None, kept=None, count=None), B.RAD_OK),
    (dict(heads=0, w=None), B.RAD_OK),
])
def test_select_refusals(kw, rc):
    assert select(**kw) == rc


IN_PLACE = dict(table=None, pages=0)


@pytest.mark.parametrize("kw,rc", [
    (dict(b=dict(seqs=-1)), B.RAD_E_SHAPE), (dict(b=dict(max_pages=-1)), B.RAD_E_SHAPE), (dict(entries=-1), B.RAD_E_SHAPE),
    (dict(pages=-1), B.RAD_E_SHAPE), (dict(lists=3), B.RAD_E_SHAPE), (dict(lists=0), B.RAD_E_SHAPE),
    (dict(to=dict(heads=4)), B.RAD_E_SHAPE), (dict(to=dict(D=64)), B.RAD_E_SHAPE), (dict(to=dict(page=48)), B.RAD_E_SHAPE),
    (dict(b=dict(seqs=1 << 22)), B.RAD_E_RANGE), (dict(entries=1 << 30), B.RAD_E_RANGE), (dict(pages=1 << 25), B.RAD_E_RANGE),
    (dict(IN_PLACE, entries=B.RAD_KV4_MOVE_MAX + 1), B.RAD_E_RANGE), (dict(IN_PLACE, to=dict()), B.RAD_E_NULL),
    (dict(table=None), B.RAD_E_NULL), (dict(src=None), B.RAD_E_NULL), (dict(count=None), B.RAD_E_NULL),
    (dict(b=dict(n=None)), B.RAD_E_NULL), (dict(b=dict(table=None)), B.RAD_E_NULL), (dict(to=dict(v=None)), B.RAD_E_NULL),
    (dict(src=P[7] + 2), B.RAD_E_ALIGN), (dict(count=P[8] + 1), B.RAD_E_ALIGN), (dict(table=P[9] + 2), B.RAD_E_ALIGN),
    (dict(start=P[10] + 2), B.RAD_E_ALIGN), (dict(to=dict(k=P[11] + 8)), B.RAD_E_ALIGN),
    (dict(src=P[0] + 64), B.RAD_E_ALIAS), (dict(count=P[1]), B.RAD_E_ALIAS), (dict(start=P[3]), B.RAD_E_ALIAS),
    (dict(table=P[2] + 4), B.RAD_E_ALIAS), (dict(to=dict(k=P[0] + 64)), B.RAD_E_ALIAS), (dict(to=dict(k=P[2])), B.RAD_E_ALIAS),
    (dict(to=dict(k=P[0], page=32)), B.RAD_E_ALIAS), (dict(IN_PLACE, src=P[2]), B.RAD_E_ALIAS),
    (dict(b=dict(seqs=0), src=None, count=None), B.RAD_OK), (dict(entries=0, src=None), B.RAD_OK),
    (dict(pages=0), B.RAD_OK),
])
def test_move_refusals(kw, rc):
    assert move(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=3), B.RAD_E_FMT), (dict(D=96), B.RAD_E_SHAPE), (dict(D=512), B.RAD_E_SHAPE), (dict(seqs=-1), B.RAD_E_SHAPE),
    (dict(rows=-1), B.RAD_E_SHAPE), (dict(max_q=-1), B.RAD_E_SHAPE), (dict(heads=0), B.RAD_E_SHAPE), (dict(qk=0), B.RAD_E_SHAPE),
    (dict(qk=3), B.RAD_E_SHAPE), (dict(ldq=255), B.RAD_E_SHAPE), (dict(ldk=0), B.RAD_E_SHAPE), (dict(ldv=511), B.RAD_E_SHAPE),
    (dict(start=None), B.RAD_E_SHAPE), (dict(seqs=1 << 22), B.RAD_E_RANGE), (dict(rows=1 << 22), B.RAD_E_RANGE),
    (dict(heads=2048, qk=2048, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20), B.RAD_E_RANGE), (dict(ldq=1 << 31), B.RAD_E_RANGE),
    (dict(seqs=1 << 21), B.RAD_E_RANGE), (dict(scale=NAN), B.RAD_E_RANGE), (dict(scale=INF), B.RAD_E_RANGE),
    (dict(q=None), B.RAD_E_NULL), (dict(k=None), B.RAD_E_NULL), (dict(v=None), B.RAD_E_NULL), (dict(g=None), B.RAD_E_NULL),
    (dict(o=None), B.RAD_E_NULL), (dict(q=P[0] + 8), B.RAD_E_ALIGN), (dict(k=P[1] + 4), B.RAD_E_ALIGN),
    (dict(v=P[2] + 2), B.RAD_E_ALIGN), (dict(g=P[3] + 2), B.RAD_E_ALIGN), (dict(start=P[4] + 1), B.RAD_E_ALIGN),
    (dict(s=P[5] + 8), B.RAD_E_ALIGN), (dict(so=P[6] + 4), B.RAD_E_ALIGN), (dict(o=P[7] + 8), B.RAD_E_ALIGN),
    (dict(ldq=260), B.RAD_E_ALIGN), (dict(ldk=257, dt=F32), B.RAD_E_ALIGN), (dict(ldv=516), B.RAD_E_ALIGN),
    (dict(o=P[0]), B.RAD_E_ALIAS), (dict(o=P[5] + 64), B.RAD_E_ALIAS), (dict(so=P[5] + 16), B.RAD_E_ALIAS),
    (dict(so=P[2]), B.RAD_E_ALIAS), (dict(so=P[7]), B.RAD_E_ALIAS), (dict(o=P[4]), B.RAD_E_ALIAS), (dict(so=P[3]), B.RAD_E_ALIAS),
    (dict(seqs=0, rows=0, q=None, k=None, v=None, g=None, o=None, s=None, so=None, start=None), B.RAD_OK),
])
def test_linear_refusals(kw, rc):
    assert linear(**kw) == rc


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 4, 64)
    with pytest.raises(TypeError, match="GPU tensor"):
        B.linear_attn(x, x, x, torch.zeros(4))
