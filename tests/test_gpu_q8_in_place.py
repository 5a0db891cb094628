"""Rotating appends to the 8-bit cache whose queries are rotated in place."""
import pytest

import sparse_paged_kv_score_gb300 as spkv
from helpers import host_bits
from test_gpu_q8 import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (32, 2), (16, 1), (40, 8)])
@pytest.mark.parametrize("past,lens,pad", [([70], [1], 0), ([5, 0, 200] * 20, [1] * 60, 0), ([7, 100, 0, 61], [40, 0, 17, 66], 3),
                                           ([0, 33], [1500, 901], 5)])
def test_queries_in_place(Hq, Hk, past, lens, pad):
    """q_out may be q itself where that is contiguous: few rows (a CTA a kv head) and many (query heads in CTAs of their own)
    give what they give into another tensor, and rows of no request are left alone."""
    b = Batch(past, lens, Hq, Hk, seed=Hq, pad=pad)
    want = b.expect()
    if pad:
        want[-pad:] = host_bits(b.qd)[-pad:]
    b.q_out = b.qd
    b.call()
    assert spkv.get_device_error(b.cache) == (0, 0)
    b.check(want)
