"""The token mixers' Python calls on the CPU: what they keep between calls.  The library's sizes are its own; addresses are fake and
nothing is enqueued."""
import os

import pytest

from rotated_w8a8_int8_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="librad.so not built")


class Emptied(dict):
    """A dict that another thread empties as soon as something is put into it."""

    def __setitem__(self, key, value):
        super().__setitem__(key, value)
        self.clear()


def test_sizes_kept_by_one_thread_may_be_cleared_by_another(monkeypatch):
    import torch
    asked = []
    monkeypatch.setattr(B, "_linear_bytes", Emptied())
    monkeypatch.setattr(B, "_values", lambda t, name: B.RAD_DT_BF16)
    monkeypatch.setattr(B, "_rows_apart", lambda t, dtype, shape, index, name: (4096, shape[1] * shape[2]))
    monkeypatch.setattr(B, "_ptr", lambda t, dtype, shape, ref, name: 4096)
    monkeypatch.setattr(B, "_workspace", lambda workspace, n, ref: asked.append(n) or (None, 0, None))
    monkeypatch.setattr(B, "_enqueue", lambda *a: None)
    x, start = torch.zeros((2000, 4, 128), dtype=torch.bfloat16), torch.tensor([0, 2000], dtype=torch.int32)
    for _ in range(2):
        B.linear_attn(x, x, x, torch.zeros(4), q_start=start, o=x)
    assert len(asked) == 2 and asked[0] == asked[1] > 0
