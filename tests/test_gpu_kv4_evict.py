"""GPU: rad_kv4_select against the oracle, bit for bit, and rad_kv4_move against moves on the host, every byte of the
cache compared; in place and to other pages and caches."""
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


def make_weights(rng, kind, shape):
    if kind == "spread":
        return (rng.random(shape) ** 8 * np.exp(rng.uniform(-30, 5, shape))).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    if kind == "close":                                       # neighbours in the last bits
        return (np.float32(1.0).view(np.uint32) + rng.integers(0, 300, shape).astype(np.uint32)).view(np.float32)
    w = rng.standard_normal(shape).astype(np.float32)        # "odd": signs, zeros of both signs, infinities, NaN
    w[rng.random(shape) < 0.2] = 0.0
    w[rng.random(shape) < 0.2] = -0.0
    w[rng.random(shape) < 0.05] = np.inf
    w[rng.random(shape) < 0.05] = -np.inf
    w[rng.random(shape) < 0.1] = np.nan
    return w


def run_select(torch, seq_len, heads, budget, first, recent, kind, seed=0, width=None, page=32):
    rng = np.random.default_rng(seed)
    seq_len = np.array(seq_len)
    width = max(1, int(max(seq_len.max(), 1) + page - 1) // page) if width is None else width
    n = width * page
    w = make_weights(rng, kind, (len(seq_len), heads, n))
    batch = C.device_batch(torch, np.zeros((len(seq_len), width), np.int32), seq_len, None, len(seq_len))
    kept = torch.full((len(seq_len), heads, budget), -7, dtype=torch.int32, device="cuda")
    kw = torch.full((len(seq_len), heads, budget + seed % 3), 77.0, device="cuda")
    _, count, _ = B.kv4_select(batch, C.put(torch, w), budget, first, recent, kept=kept, kept_weight=kw)
    kept, kw, count = kept.cpu().numpy(), kw.cpu().numpy(), count.cpu().numpy()
    for b, L in enumerate(np.clip(seq_len, 0, n)):
        assert count[b] == min(L, budget)
        for h in range(heads):
            want = X.select(w[b, h], int(L), budget, first, recent)
            assert np.array_equal(kept[b, h, :len(want)], want), (b, h, L)
            assert np.all(kept[b, h, len(want):] == -7)
            assert np.array_equal(kw[b, h, :len(want)].view(np.uint32), w[b, h, want].view(np.uint32))
            assert np.all(kw[b, h, len(want):] == 77.0)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "close", "odd"])
@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (7, 0, 0), (64, 4, 16), (64, 32, 32), (300, 0, 299), (1000, 3, 9)])
def test_select(torch, budget, first, recent, kind):
    print("select", budget, first, recent, kind, flush=True)
    run_select(torch, [0, 1, 6, 64, 65, 300, 1001, 777, -3], 3, budget, first, recent, kind, seed=budget)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("L,budget", [(4096, 1024), (16385, 4000), (40000, 129), (70001, 65000), (199999, 16384)])
def test_select_of_long_sequences(torch, L, budget, kind):
    print("long", L, budget, kind, flush=True)
    run_select(torch, [L, L // 3, 17], 2, budget, 4, budget // 5, kind, seed=L)


def test_select_of_many_sequences(torch):
    rng = np.random.default_rng(1)
    run_select(torch, rng.integers(0, 400, 700), 2, 100, 2, 30, "spread", seed=2)


def test_select_of_many_long_sequences(torch):
    # more (sequence, head) pairs than slices are wanted for
    rng = np.random.default_rng(6)
    n, L, heads, budget = 550, 66048, 2, 500
    w = torch.rand((n, heads, L), device="cuda")
    seq_len = rng.integers(60000, L + 1, n)
    batch = C.device_batch(torch, np.zeros((n, L // 32), np.int32), seq_len, None, n)
    kept, count, kw = B.kv4_select(batch, w, budget, 2, 30)
    assert torch.all(count == budget)
    for b in (0, 17, 311, n - 1):
        for h in range(heads):
            x = w[b, h].cpu().numpy()
            want = X.select(x, int(seq_len[b]), budget, 2, 30)
            assert np.array_equal(kept[b, h].cpu().numpy(), want) and np.array_equal(kw[b, h, :budget].cpu().numpy(), x[want])
    # every list ascends, and its least weight is no less than what a sort puts there
    assert torch.all(kept[..., 1:] > kept[..., :-1])


def test_lengths_past_the_room_are_cut_to_it(torch):
    run_select(torch, [500, 96, 97], 1, 20, 1, 2, "spread", seed=4, width=3)


# ------------------------------------------------------------------------------------------------ move --

def same_cache(got, want):
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        a, b = getattr(got, name).cpu().numpy(), getattr(want, name)
        if a.dtype == np.float16:
            a, b = a.view(np.uint16), b.view(np.uint16)
        assert np.array_equal(a, b), name


def run_move(torch, seq_len, source, count, heads, D, page, to_start=None, to_page=None, to_len=None, seed=0, edit=None, edit_to=None):
    """source [B][lists][n]; to_page None: in place; `to_len` tokens of room in the other cache's tables."""
    rng = np.random.default_rng(seed)
    seq_len = np.array(seq_len)
    table, pages = C.page_table(rng, np.maximum(seq_len, 1), page, None)
    if edit is not None:
        edit(table, pages)
    ref = O.Cache(pages, heads, page, D, rng)
    dev = C.device_cache(torch, ref)
    batch = C.device_batch(torch, table, seq_len, None, len(seq_len))
    source = np.asarray(source, np.int32)
    src = C.put(torch, source[:, 0] if source.shape[1] == 1 else source)
    cnt = C.put(torch, np.asarray(count, np.int32))
    ts = None if to_start is None else C.put(torch, np.asarray(to_start, np.int32))
    start = np.zeros(len(seq_len), np.int64) if to_start is None else to_start
    if to_page is None:
        B.kv4_move(dev, batch, src, cnt, to_start=ts)
        X.move(ref, table, seq_len, source, count, ref, table, start)
        same_cache(dev, ref)
        return
    to_table, to_pages = C.page_table(rng, np.full(len(seq_len), to_len), to_page, None)
    if edit_to is not None:
        edit_to(to_table, to_pages)
    other = O.Cache(to_pages, heads, to_page, D, rng)
    dev_to = C.device_cache(torch, other)
    B.kv4_move(dev, batch, src, cnt, to=dev_to, to_table=C.put(torch, to_table), to_start=ts)
    X.move(ref, table, seq_len, source, count, other, to_table, start)
    same_cache(dev_to, other)
    same_cache(dev, ref)


@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("page,to_page", [(32, 32), (64, 256), (128, 32)])
def test_lists_a_head_to_other_pages(torch, D, page, to_page):
    rng = np.random.default_rng(D + page)
    lens = [300, 40, 0, 129]
    src = np.stack([np.stack([np.sort(rng.choice(max(n, 100), 100, replace=False)) for _ in range(3)]) for n in lens])
    run_move(torch, lens, src, [100, 37, 100, 200], 3, D, page, [0, 5, 3, 250], to_page, 320, seed=D)


def test_any_order_repeats_and_entries_that_are_no_token(torch):
    rng = np.random.default_rng(4)
    src = rng.integers(-20, 320, (3, 2, 333))
    run_move(torch, [300, 120, 7], src, [333, 333, -5], 2, 128, 64, [1, 2, 3], 32, 350, seed=4)
    run_move(torch, [300, 120, 7], src[:, :1], [330, 9, 1], 2, 64, 32, None, 64, 100, seed=5)     # past the table


def test_absent_pages_give_and_take_nothing(torch):
    def edit(table, pages):
        table[0, 1], table[1, 0] = -1, pages + 4

    def edit_to(table, pages):
        table[0, 0], table[1, 2] = pages, -9
    rng = np.random.default_rng(5)
    run_move(torch, [300, 120], rng.integers(0, 300, (2, 2, 150)), [150, 150], 2, 128, 64, [0, 60], 64, 250, seed=5, edit=edit, edit_to=edit_to)


@pytest.mark.parametrize("start", [[-3, -1 << 31, (1 << 31) - 1], [1 << 30, 333, 349], [-10, -200, 0]])
def test_targets_outside_the_table_take_nothing(torch, start):
    rng = np.random.default_rng(6)
    run_move(torch, [300, 120, 44], rng.integers(0, 300, (3, 1, 50)), [50, 50, 50], 2, 64, 32, start, 32, 350, seed=6)
    run_move(torch, [300, 120, 44], rng.integers(0, 300, (3, 1, 50)), [50, 50, 50], 2, 64, 32, start, seed=7)


@pytest.mark.parametrize("D", B.KV_HEAD_DIMS)
@pytest.mark.parametrize("page", [32, 128])
def test_accepted_paths_in_place(torch, D, page):
    # ascending paths of a drafted tree, to the front of its tokens
    rng = np.random.default_rng(D)
    lens, drafted = [300, 64, 70, 33], [60, 64, 1, 0]
    src, count = np.zeros((4, 1, 64), np.int64), [13, 64, 1, 0]
    for b, (n, d) in enumerate(zip(lens, drafted)):
        src[b, 0, :count[b]] = n - d + np.sort(rng.choice(max(d, 1), count[b], replace=False))
    run_move(torch, lens, src, count, 3, D, page, [n - d for n, d in zip(lens, drafted)], seed=D)


def test_in_place_reads_all_before_it_writes(torch):
    rng = np.random.default_rng(9)
    n = B.RAD_KV4_MOVE_MAX
    for start in (0, 3, 7):
        src = np.stack([np.stack([start + rng.permutation(n) for _ in range(2)]) for _ in range(3)])
        run_move(torch, [n + 40] * 3, src, [n, n - 1, 100], 2, 128, 64, [start] * 3, seed=start)
    run_move(torch, [n], np.arange(n)[None, None, ::-1], [n], 2, 256, 32, None, seed=3)


def test_to_other_pages_of_the_same_cache(torch):
    rng = np.random.default_rng(2)
    ref = O.Cache(12, 2, 32, 64, rng)
    table, to_table = np.array([[3, 1, 7], [0, 9, 2]], np.int32), np.array([[5, 11], [6, 4]], np.int32)
    dev, seq_len = C.device_cache(torch, ref), np.array([90, 61])
    batch = C.device_batch(torch, table, seq_len, None, 2)
    src = np.stack([np.stack([np.sort(rng.choice(n, 40, replace=False)) for _ in range(2)]) for n in seq_len]).astype(np.int32)
    B.kv4_move(dev, batch, C.put(torch, src), C.put(torch, np.array([40, 40], np.int32)), to_table=C.put(torch, to_table))
    X.move(ref, table, seq_len, src, [40, 40], ref, to_table, [0, 0])
    same_cache(dev, ref)
