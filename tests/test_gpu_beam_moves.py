"""beam_reorder where nothing has to be copied, against what was there before the call."""
import numpy as np
import pytest
import torch

import sparse_paged_kv_score_gb300 as spkv
from test_gpu_beam import FORMATS, Beams

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sums", [True, False])
@pytest.mark.parametrize("by", [0, 1, 4])
def test_own_parents_and_rotations(fmt, sums, by):
    """Every beam its own parent: nothing changes.  Beams that only change places: their whole table rows do, up to the
    part-filled page, and no pool, sum or count changes."""
    W = 6
    s = Beams(fmt, 2, W, 2, [200, 77], seed=by, sums=sums)
    table, pools = s.table.clone(), [p.clone() for p in s.pools]
    ksum, cnt = (None, None) if not sums else (s.ksum.clone(), s.cnt_d.clone())
    parents = np.tile((np.arange(W) + by) % W, (2, 1))
    s.call(parents)
    assert spkv.get_device_error(s.cache) == (0, 0)
    want = table.clone()
    for b, L in enumerate((200, 77)):
        for w in range(W):
            n = L // 64 + 1
            want[b * W + w, :n] = table[b * W + parents[b, w], :n]
    assert torch.equal(s.table, want)
    assert by or torch.equal(s.table, table)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(s.pools, pools))
    if sums:
        assert torch.equal(s.ksum, ksum) and torch.equal(s.cnt_d, cnt)
