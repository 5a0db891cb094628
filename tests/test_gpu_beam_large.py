"""beam_select with more groups than there are warps at once (stages used again, steps from row to row, ended beams between
live ones), and with as many of a request as it takes."""
import numpy as np
import pytest
import torch

import sparse_paged_kv_score_gb300 as spkv
from test_gpu_beam import Select, cums, logits, small_cache

pytestmark = pytest.mark.gpu


def rounds(B, W, V, size):
    """Groups of 4 KiB of all rows to a warp of the first kernel, of whose there are 24 on an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return B * W * -(-V * size // 4096) / (24 * sms)


LARGE = [
    pytest.param(torch.bfloat16, 32, 8, 128256, 16, 0, 0, id="bf16"),
    pytest.param(torch.float32, 32, 8, 50021, 9, 3, 5, id="fp32 odd, rows apart"),
    pytest.param(torch.float16, 64, 8, 45001, 5, 1, 3, id="fp16 odd, rows apart"),
    pytest.param(torch.float32, 1100, 4, 3001, 4, 0, 1, id="short rows"),
]


@pytest.mark.parametrize("dtype,B,W,V,K,pad,shift", LARGE)
@pytest.mark.parametrize("ended", [0.0, 0.3, 0.9])
def test_many_groups_a_warp(dtype, B, W, V, K, pad, shift, ended):
    """Against the 64-bit form; ended beams' logits are NaN, which nothing may read.  A call of one request by itself, whose
    groups have a warp each, gives the same bits, and so does the whole call again."""
    assert rounds(B, W, V, 4 if dtype == torch.float32 else 2) > 2.9
    x, cum = logits(B, W, V, dtype, seed=V), cums(B, W, V)
    gone = np.random.default_rng(V).random((B, W)) < ended
    if ended:
        gone[0, 0] = gone[B - 1, W - 1] = True
        gone[B // 2] = True
    cum[gone] = -np.inf
    x[torch.from_numpy(gone)] = float("nan")
    s = Select(x, cum, K, pad=pad, shift=shift)
    s.call()
    t, p, v = s.check()
    assert not gone[np.arange(B)[:, None], p][p >= 0].any()
    s.call()
    assert np.array_equal(s.tokens.cpu().numpy(), t) and np.array_equal(s.scores.cpu().numpy().astype(np.float64), v)
    plan = spkv.BeamPlan(s.cache, W, V)
    one = [torch.empty(1, K, dtype=d, device=s.tokens.device) for d in (torch.int32, torch.int32, torch.float32)]
    for b in (0, 1, B // 2, B - 1):
        spkv.beam_select(s.cache, plan, s.x[b:b + 1], s.cum_d[b:b + 1], *one)
        assert torch.equal(one[0][0], s.tokens[b]) and torch.equal(one[1][0], s.parents[b]) and torch.equal(one[2][0], s.scores[b])


@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("B,W,V", [(2, 64, 140001), (1, 64, 512 * 1024)])
def test_many_groups_of_a_request(B, W, V, alike):
    """More group keys than the selection's own room (8192), up to the most that it takes (32768); with all logits alike the
    lists overflow and everything is searched for."""
    K = 128
    if alike:
        x, cum = torch.zeros(B, W, V), np.full((B, W), -1.0, np.float32)
        cum[:, 0] = -np.inf
    else:
        x, cum = logits(B, W, V, torch.float32, seed=W), cums(B, W, W)
        cum[:, 5] = -np.inf
    assert W * -(-V * 4 // 4096) in (8768, 32768)
    s = Select(x, cum, K, cache=small_cache())
    s.call()
    t, p, _ = s.check()
    if alike:
        assert np.array_equal(t, np.tile(np.arange(K), (B, 1))) and np.all(p == 1)
