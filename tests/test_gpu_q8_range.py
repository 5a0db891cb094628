"""Values as large as the attention over the 8-bit cache takes."""
import numpy as np
import pytest

import q8_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from test_gpu_q8 import Cache, check, queries, u8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("pages,e", [(64, 100), (2, 105), (1, 106), (2, -110)])
def test_largest_values(G, pages, e):
    """Values of nearly 2^(e + 1): weights reach 2^15 of the running reference, so sums of N
    tokens stay in fp32 up to N |v| = 2^113.  The later half's scores lie 7.9 log2 units above the first half's, as far as the
    reference lets them rise."""
    c = Cache(1, 1, pages, [64 * pages], seed=e % 100, junk=False, sums=False)
    rng = np.random.default_rng(G)
    qx, q = queries(1, G, seed=9)
    qx = np.broadcast_to(qx[:, :1], qx.shape).copy()      # one query, whatever the heads
    q[:] = q[:, :1].clone()
    k = np.zeros((1, c.n_phys, 64, 128), np.float32)
    up = 7.9 * np.log(2) * np.sqrt(128) / (qx[0, 0].astype(np.float64) ** 2).sum()
    late = 64 * pages // 2                                 # tokens before the rise
    for p in range(pages):
        k[0, c.pt[0, p], min(64, max(0, late - 64 * p)):] = qx[0, 0] * up
    v = (1 + rng.random(k.shape)) * np.where(rng.random(k.shape) < 0.9, 1, -1) * 2.0 ** e
    c.blob[:] = ref.pool_of(k, np.minimum(v, 1.99 * 2.0 ** e).astype(np.float32))
    c.pool.copy_(u8(c.blob))
    sel = np.arange(pages)[None, None]
    n = np.full((1, 1), pages)
    out, lse = c.attend(q, sel, n)
    want = ref.attention(qx, c.blob, c.pt, sel, n, c.L)
    assert np.isfinite(out.cpu().numpy()).all() and 64 * pages * 2.0 ** (e + 1) <= 2.0 ** 113
    check(out, lse, want)
    assert spkv.get_device_error(c.handle) == (0, 0)
