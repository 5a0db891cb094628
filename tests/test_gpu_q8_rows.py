"""Attention over the 8-bit cache against attention over the rows that went into it, in 64 bits."""
import numpy as np
import pytest
import torch

import q8_ref as ref
import sparse_paged_kv_score_gb300 as spkv
from helpers import DEV, bf, f32, i32
from q4_ref import bf16, bf16_bits

pytestmark = pytest.mark.gpu


def attend(k, v, q):
    """(out, lse, pool bytes, kernel's error bounds) of one request whose rows k, v [L][Hk][128] (bf16 numbers) are appended as
    they are, for the query heads q [Hq][128] over all pages."""
    L, Hk, Hq = k.shape[0], k.shape[1], q.shape[0]
    n = -(-L // 64)
    pool = torch.zeros(Hk, n, ref.BLOB, dtype=torch.uint8, device=DEV)
    cache = spkv.paged_kv_create_q8(pool, torch.zeros(Hk, n, 4, 128, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV))
    table, lens = i32(np.arange(n)[None]), i32([L])
    spkv.paged_kv_append_rope(cache, bf(bf16_bits(k)), bf(bf16_bits(v)), lens, table, row_first=i32([0, L]))
    sel, n_sel = i32(np.tile(np.arange(n), (1, Hk, 1))), i32(np.full((1, Hk), n))
    out, lse = torch.zeros(1, Hq, 128, device=DEV), torch.zeros(1, Hq, device=DEV)
    spkv.sparse_decode_attn(cache, bf(bf16_bits(q))[None], table, sel, n_sel, lens, out, lse)
    assert spkv.get_device_error(cache) == (0, 0)
    blob = pool.cpu().numpy()
    _, _, e_out, e_lse = ref.attention(q[None].astype(np.float64), blob, np.arange(n)[None], np.tile(np.arange(n), (1, Hk, 1)),
                                       np.full((1, Hk), n), np.array([L]))
    return out[0].cpu().numpy(), lse[0].cpu().numpy(), blob, e_out[0], e_lse[0]


def scales_of(blob, h, L, keys):
    return np.repeat(ref.scales(blob[h], keys).astype(np.float64), 16, -1).reshape(-1)[:L]


@pytest.mark.parametrize("L,Hk,G", [(1, 2, 1), (15, 1, 4), (64, 2, 4), (193, 1, 8), (1000, 2, 16), (4160, 1, 4)])
def test_attention_is_that_of_the_rows_but_for_half_a_step_of_the_codes(L, Hk, G):
    """A key's dims are off by s / 2 at most, so a score by d = sum |q| s / 2 / sqrt(128), a weight by a factor within
    e^(+- 2 d) (its own and the sum's), and a value by its own s / 2; the kernel's error over the values that are held comes
    on top."""
    rng = np.random.default_rng(L)
    size = 2.0 ** rng.integers(-2, 3, (L, Hk, 1))
    k, v = (bf16(rng.standard_normal((L, Hk, 128)) * x) for x in (0.3 * size, size[::-1]))
    q = bf16(rng.standard_normal((Hk * G, 128)))
    out, lse, blob, e_out, e_lse = attend(k, v, q)
    for h in range(Hk):
        ks, vs = (scales_of(blob, h, L, keys) for keys in (True, False))
        for g in range(h * G, h * G + G):
            x = k[:, h].astype(np.float64) @ q[g].astype(np.float64) / np.sqrt(128)
            p = np.exp(x - x.max())
            want = p @ v[:, h].astype(np.float64) / p.sum()
            d = np.abs(q[g].astype(np.float64)).sum() * ks.max() / 2 / np.sqrt(128)
            bound = vs.max() / 2 + np.expm1(2 * d) * np.abs(v[:, h]).max() + e_out[g]
            assert np.abs(out[g] - want).max() <= bound
            assert abs(lse[g] - (x.max() + np.log(p.sum()))) <= d + e_lse[g]


@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("sign", [1, -1])
def test_bf16_values_come_out_half_a_step_of_theirs_high(G, sign):
    """Equal weights over all 128 bf16 numbers of a binade, in every dim: the output is their mean and half their distance."""
    t, d = np.arange(128)[:, None, None], np.arange(128)
    v = (sign * (1 + (t + d) % 128 / 128)).astype(np.float32)
    out, lse, _, e_out, e_lse = attend(np.zeros((128, 1, 128), np.float32), v, np.zeros((G, 128), np.float32))
    want = v[:, 0].astype(np.float64).mean(0) + 2.0 ** -8
    assert np.all(np.abs(out - want).max(-1) <= e_out) and e_out.max() < 2.0 ** -12
    assert np.all(np.abs(lse - np.log(128)) <= e_lse)
