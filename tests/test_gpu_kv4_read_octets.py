"""GPU: the read-back of many rows, which takes octets of tokens, against the same rows read a few at a time: bit for bit, and what
is not read left as it was."""
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


def read(torch, cache, table, seq_len, start, rows):
    k, v = (torch.full((rows, cache.heads, cache.D), 55.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.kv4_read(cache, C.device_batch(torch, table, seq_len, start, rows), k, v)
    return k.view(torch.int16), v.view(torch.int16)


@pytest.mark.parametrize("page", [32, 256])
@pytest.mark.parametrize("D,heads,new,ctx", [
    (128, 8, [6500], [3]), (128, 3, [9000, 0, 5003, 4100, 1], [7, 50, -4, 0, 5]), (128, 2, [15001, 11000], [13, -20]),
    (256, 8, [1700, 1500], [1, 8]), (256, 2, [13000], [-1001]), (128, 1, [20000] * 6 + [20003, 11111], [1, 2, 3, 4, 5, 6, 7, -8]),
    (64, 8, [4001, 4000, 5000, 3999, 0, 4100, 4007, 4008, 4009, 17], [0, 3, 5, 8, 9, -2, 100, 6, 1, 20])])
def test_read_back_of_many_rows(torch, D, heads, new, ctx, page):
    rng = np.random.default_rng(D + heads)
    seq_len, start = np.array(new) + np.array(ctx), C.ragged(new)
    table, pages = C.page_table(rng, np.maximum(seq_len, 0), page)
    table[0, 1], table[0, 4] = -1, pages + 2                   # absent pages
    ref = O.Cache(pages, heads, page, D, rng)
    ref.k_scale[:] = rng.uniform(0.1, 2, ref.k_scale.shape).astype(np.float16)
    ref.v_scale[:] = rng.uniform(0.1, 2, ref.v_scale.shape).astype(np.float16)
    cache, T = C.device_cache(torch, ref), int(start[-1]) + 5
    k, v = read(torch, cache, table, seq_len, start, T)
    few = 4000 if heads == 1 else 400
    for b, n in enumerate(new):
        for lo in range(0, n, few):
            m = min(few, n - lo)
            length = int(seq_len[b]) - (n - lo - m)           # rows lo .. lo + m - 1 as the last of a shorter sequence
            if length <= 0:
                want = [torch.full((m, heads, D), 55.0, dtype=torch.bfloat16, device="cuda").view(torch.int16)] * 2
            else:
                want = read(torch, cache, table[b:b + 1], [length], np.array([0, m], np.int32), m)
            for got, w in zip((k, v), want):
                assert torch.equal(got[start[b] + lo:start[b] + lo + m], w), (b, lo)
    for got in (k, v):
        assert torch.all(got[start[-1]:].view(torch.bfloat16) == 55.0)
