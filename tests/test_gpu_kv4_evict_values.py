"""GPU: selection where no place is left for weights to compete for (the first and the recent tokens fill the budget), whatever
the weights are, more of one kind than the kernel holds in LDS among them; and from lists of millions of tokens."""
import numpy as np
import pytest

import layer_cases as C
from oracle import mixers as X
from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    return _t


@pytest.mark.parametrize("fill", [np.nan, -np.inf, 0.0, 1.0])
@pytest.mark.parametrize("L,room", [(5000, 5024), (20000, 20000), (65530, 65536), (70000, 80000)])
def test_budgets_that_first_and_recent_tokens_fill(torch, L, room, fill):
    print("no place left", L, room, fill, flush=True)
    rng = np.random.default_rng(L)
    w = np.full((2, 2, room), fill, np.float32)
    w[1] = np.where(rng.random(w[1].shape) < 0.9, fill, rng.standard_normal(w[1].shape)).astype(np.float32)
    batch = C.device_batch(torch, np.zeros((2, 1), np.int32), [L, L - 77], None, 2)
    for first, recent in ((0, 64), (40, 60), (100, 0)):
        budget = first + recent
        kept, count, kw = B.kv4_select(batch, C.put(torch, w), budget, first, recent)
        assert count.tolist() == [budget] * 2
        for b, n in enumerate((L, L - 77)):
            want = X.select(w[b, 0], n, budget, first, recent)
            for h in range(2):
                assert np.array_equal(kept[b, h].cpu().numpy(), want)
                assert np.array_equal(kw[b, h, :budget].cpu().numpy(), w[b, h, want], equal_nan=True)


@pytest.mark.parametrize("L", [1048580, 1560000, 1600001, 5000000])
def test_lists_of_many_slices(torch, L):
    print("slices", L, flush=True)
    rng = np.random.default_rng(L)
    w = (rng.random((2, 1, (L + 3) // 4 * 4)) ** 8).astype(np.float32)
    seq_len = [L, L // 2]
    kept, count, kw = B.kv4_select(C.device_batch(torch, np.zeros((2, 1), np.int32), seq_len, None, 2), C.put(torch, w), 2000, 4, 300)
    for b, n in enumerate(seq_len):
        want = X.select(w[b, 0], n, 2000, 4, 300)
        assert np.array_equal(kept[b, 0].cpu().numpy(), want) and np.array_equal(kw[b, 0, :2000].cpu().numpy(), w[b, 0, want])
