"""GPU: rad_kv4_append_at against the oracle, codes, scales and turned queries bit for bit: positions that repeat, that lie
apart from the place in the cache, and that the table does not have (their rows are skipped)."""
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


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("new,ctx", [([1, 1, 1, 1], [40, 0, 7, 95]), ([5, 1, 16, 0, 9], [33, 64, 7, 3, -4]), ([150], [20])])
@pytest.mark.parametrize("D,rot,dim,style", [(64, False, 64, 0), (128, True, 128, 1), (256, True, 64, 0)])
def test_positions_of_their_own(torch, D, rot, dim, style, new, ctx, dtype):
    rng = np.random.default_rng(D + sum(new))
    H, HQ, page, table_rows = 2, 3, 32, 50
    start, T, seq_len = C.ragged(new), sum(new) + 2, np.array(new) + np.array(ctx)
    one = all(n == 1 for n in new)
    T = sum(new) if one else T
    table, pages = C.page_table(rng, np.maximum(seq_len, 0), page)
    ref = O.Cache(pages, H, page, D, rng)
    dev = C.device_cache(torch, ref)
    x = O.to_dtype(rng.standard_normal((T, HQ + 2 * H, D)), dtype)
    tab = C.rope_table(table_rows, dim)
    position = rng.integers(0, table_rows, T).astype(np.int32)
    position[rng.random(T) < 0.2] = table_rows                   # the table ends before it
    position[rng.random(T) < 0.1] = -1
    q, k, v = C.put(torch, x, dtype).split([HQ, H, H], dim=1)
    q_out = torch.full((T, HQ, D), 77.0, dtype=C.torch_dtype(torch, dtype), device="cuda")
    B.kv4_append(dev, C.device_batch(torch, table, seq_len, None if one else start, T), k, v, q, rope=C.put(torch, tab), rope_style=style,
                 rotate=rot, q_out=q_out, position=C.put(torch, position))
    want = np.full((T, HQ, D), 77.0, np.float32)
    for b, n in enumerate(new):
        for i in range(n):
            row, t = int(start[b]) + i, int(seq_len[b]) - n + i
            if t < 0 or not 0 <= position[row] < table_rows:
                continue
            q1, k1, v1 = O.append_f32(x[row:row + 1, :HQ], x[row:row + 1, HQ:HQ + H], x[row:row + 1, HQ + H:],
                                      tab[position[row]][None], style, rot)
            want[row] = O.to_dtype(q1[0], dtype)
            ref.put(int(table[b, t // page]), t % page, (k1[0][0], k1[1][0]), (v1[0][0], v1[1][0]))
    assert np.array_equal(C.host(q_out), want)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        a, b = getattr(dev, name).cpu().numpy(), getattr(ref, name)
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8)), name
