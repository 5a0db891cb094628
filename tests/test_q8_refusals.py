"""What the 8-bit cache refuses on the host, before any CUDA call, and what its handle launches."""
import ctypes
import json

import numpy as np
import pytest
import torch

import fake_cuda
import q4_ref
import q8_ref as ref


@pytest.fixture(scope="module")
def lib():
    from sparse_paged_kv_score_gb300 import build
    build.build()
    from sparse_paged_kv_score_gb300 import _abi
    return _abi.load()


@pytest.fixture(scope="module")
def fake(tmp_path_factory, lib):
    return fake_cuda.build(str(tmp_path_factory.mktemp("fake")))


GOOD = dict(n_kv_heads=2, head_dim=128, page_tokens=64, subblock=16, n_phys_pages=4, kv_pool=4096, ksum=4096, page_cnt=4096,
            max_units=0, ksum_bf16=0)


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=64), "EUNSUPPORTED"), (dict(page_tokens=32), "EUNSUPPORTED"), (dict(subblock=8), "EUNSUPPORTED"),
    (dict(n_kv_heads=0), "EINVAL"), (dict(n_phys_pages=0), "EINVAL"), (dict(kv_pool=None), "EINVAL"),
    (dict(kv_pool=4104), "EINVAL"), (dict(page_cnt=None), "EINVAL"), (dict(ksum=4104), "EINVAL"),
    (dict(max_units=-1), "EINVAL"), (dict(max_units=4097), "EINVAL"), (dict(ksum_bf16=2), "EINVAL"),
    (dict(n_phys_pages=1 << 30), "EUNSUPPORTED")])
def test_descriptions(lib, bad, status):
    from sparse_paged_kv_score_gb300 import _abi
    out = ctypes.c_void_p(1)
    d = _abi.SpkvDescQ8(**{**GOOD, **bad})
    assert lib.paged_kv_create_q8(ctypes.byref(d), None, ctypes.byref(out)) == getattr(_abi, "SPKV_" + status)
    assert not out.value
    assert lib.paged_kv_create_q8(None, None, ctypes.byref(out)) == _abi.SPKV_EINVAL
    assert lib.paged_kv_create_q8(ctypes.byref(d), None, None) == _abi.SPKV_EINVAL
    assert lib.paged_kv_unpack_q8(None, 16, 1, 16, 16, None) == _abi.SPKV_EINVAL


def test_arguments():
    import sparse_paged_kv_score_gb300 as spkv
    pool = torch.zeros(2, 3, spkv.Q8_PAGE_BYTES, dtype=torch.uint8)
    with pytest.raises(ValueError, match="16416"):
        spkv.paged_kv_create_q8(pool[0], None, None)
    with pytest.raises(ValueError, match="page_cnt"):
        spkv.paged_kv_create_q8(pool, torch.zeros(2, 3, 4, 128), None)
    with pytest.raises((ValueError, TypeError)):
        spkv.paged_kv_create_q8(pool, None, None)   # not on a GPU


HANDLE = """
import ctypes, json
P = 4096
def handle8(Hk, n_phys=8):
    d = f.abi.SpkvDescQ8(Hk, 128, 64, 16, n_phys, P, P, P, 4096, 0)
    h = ctypes.c_void_p()
    assert f.lib.paged_kv_create_q8(ctypes.byref(d), None, ctypes.byref(h)) == 0
    return h
"""


def test_calls_for_other_formats_refuse_an_8bit_handle(fake):
    """SPKV_EUNSUPPORTED and nothing launched; the calls that know the format launch its kernels."""
    program = HANDLE + """
h = handle8(2)
prepared = [e.split()[1] for e in f.events() if e.startswith("set ")]
pd = f.abi.SpkvPageDir()
pd.dir, pd.dev_segs, pd.host_chunks, pd.n_dir, pd.seg_shift, pd.n_dev_segs, pd.n_host_segs = P, P, P, 1, 6, 1, 1
words = (ctypes.c_int32 * 2)(0, 1)
plan = ctypes.c_void_p()
calls = dict(
    paged_kv_append=(P, P, P, P, 1, None),
    decode_append_score=(P, P, P, 1, 8, P, 4, P, P, None),
    lazy_rope_decode_attn=(P, 1, 8, P, P, 2, P, 4, P, 1, 1e4, P, P, None),
    lazy_rope_prefill_attn=(P, 1, 2, 8, P, P, 2, P, 4, P, 1, 1e4, P, P, None),
    lazy_rope_prefill_step=(P, 1, 2, 8, P, P, 2, P, 4, P, P, 1, 1e4, P, P, None),
    lazy_alibi_prefill_attn=(P, 1, 2, 8, P, P, 2, P, 4, P, P, 1, P, P, P, None),
    attn_column_scores=(P, 1, 2, 8, P, 4, P, P, None),
    attn_column_scores_lse=(P, P, 1, 2, 8, P, 4, P, P, None),
    retrieve_pages=(P, P, 8, P, 4, 1, P, P, P, P, P, 4, 4, None),
    retrieve_pages_dir=(P, P, 8, ctypes.byref(pd), 4, 1, P, P, P, P, P, 4, 4, None),
    lazy_docs_plan_create=(1, 8, words, 1, 1, words, ctypes.byref(plan)),
    paged_kv_unpack_q4=(P, 1, P, P, None),
)
refused = {name: [getattr(f.lib, name)(h, *args), len(f.events())] for name, args in calls.items()}
own = dict(
    paged_kv_append_rope=(P, 256, P, 256, 3, 3, None, P, P, 4, None, None, 0, 0, None, None),
    paged_kv_unpack_q8=(P, 1, P, P, None),
    sparse_decode_attn=(P, 1, 8, P, 4, P, P, 4, P, P, P, None),
    sparse_decode_attn_slots=(P, 1, 8, P, P, P, 4, 4, P, P, P, None),
    sparse_decode_attn_dir=(P, 1, 8, ctypes.byref(pd), 4, P, P, 4, P, P, P, None),
    score_blocks=(P, 1, 8, P, 4, P, P, None),
)
runs = {name: [getattr(f.lib, name)(h, *args), f.events()] for name, args in own.items()}
bad = dict(
    out_4_byte=f.lib.sparse_decode_attn(h, P, 1, 8, P, 4, P, P, 4, P, P + 4, P, None),
    wide_table=f.lib.sparse_decode_attn(h, P, 1, 8, P, (1 << 25) + 1, P, P, 4, P, P, P, None),
    group=f.lib.sparse_decode_attn(h, P, 1, 34, P, 4, P, P, 4, P, P, P, None),
    unpack_8_byte=f.lib.paged_kv_unpack_q8(h, P, 1, P + 8, P, None),
    negative=f.lib.paged_kv_unpack_q8(h, P, -1, P, P, None),
)
other = [f.lib.paged_kv_unpack_q8(f.handle(q4, 2), P, 1, P, P, None) for q4 in (False, True)]
print(json.dumps([prepared, refused, runs, bad, other]))
"""
    prepared, refused, runs, bad, other = json.loads(fake_cuda.run(fake, program))
    assert len([n for n in prepared if "attn_q8" in n]) == 9 and not any("attn_q4" in n or "prefill" in n for n in prepared)
    assert all(v == [-6, 0] for v in refused.values()), refused
    for name, kernel in (("paged_kv_append_rope", "append_q8"), ("paged_kv_unpack_q8", "unpack_q8"), ("sparse_decode_attn", "attn_q8"),
                         ("sparse_decode_attn_slots", "attn_q8"), ("sparse_decode_attn_dir", "attn_q8"), ("score_blocks", "score")):
        assert runs[name][0] == 0 and len(runs[name][1]) == 1 and kernel in runs[name][1][0], name
    assert bad == dict(out_4_byte=-1, wide_table=-1, group=-6, unpack_8_byte=-1, negative=-1)
    assert other == [-6, -6]


@pytest.mark.parametrize("sms", [[152, 148], [90, 85], [40, 20, 8, 1]])
def test_launch_choices(fake, sms):
    """Attention: where CTAs take parts of units (mode 2) the grid is whole units; never more CTAs than have room at once.
    Appends: a CTA for every window and kv head, or slice of them."""
    program = HANDLE + """
import re
got, rows = [], []
for sms in SMS:
    f.rt.fake_sms(sms)
    for Hk in (1, 8):
        h = handle8(Hk)
        f.events()
        for B in (1, 2, 13, 32, 61, 128, 256, 500):
            for n in (1, 3, 4, 17, 65, 129, 700):
                for G in (1, 5, 16):
                    assert f.lib.sparse_decode_attn(h, P, B, G * Hk, P, 9, P, P, n, P, P, P, None) == 0
                    (e,) = f.events()
                    heads, mode, grid = map(int, re.search(r"attn_q8_kernelILi(\\d+)E\\S*ModeE(\\d)\\S* (\\d+)$", e).groups())
                    got.append([sms, B * Hk, G, heads, mode, grid])
        for n in (1, 5, 200, 1000, 30000):
            assert f.lib.paged_kv_append_rope(h, P, 128 * Hk, P, 128 * Hk, n, n, None, P, P, 4, None, None, 0, 0, None, None) == 0
            (e,) = f.events()
            rows.append([sms, Hk, n, "blocks" in e, int(e.split()[-1])])
print(json.dumps([got, rows]))
""".replace("SMS", repr(sms))
    got, rows = json.loads(fake_cuda.run(fake, program))
    room = {4: 3, 8: 2, 16: 2}      # CTAs of an SM
    for m, U, G, heads, mode, grid in got:
        assert heads == (4 if G <= 4 else 8 if G <= 8 else 16)
        assert 1 <= grid <= room[heads] * m, (m, U, G, mode, grid)
        assert mode != 2 or grid % U == 0
    for m, Hk, n, blocks, grid in rows:
        window = 16 if blocks else 1 if (n + 3) // 4 * Hk < m else 4
        assert grid == (n + window - 1) // window and (blocks or grid * window >= n)


def test_reference_pins():
    """The tests' own form of the format: what spkv.h says of it."""
    assert sorted(np.concatenate([ref.KC, ref.VC]).flatten()) == list(range(16384))
    rng = np.random.default_rng(0)
    x = q4_ref.bf16(rng.standard_normal((1, 3, 64, 128)) * np.exp(rng.standard_normal((1, 3, 64, 1))))
    blob = ref.pool_of(x, x)
    for keys in (True, False):
        y, s = ref.rows(blob, keys), np.repeat(ref.scales(blob, keys), 16, -1)[..., None]
        assert np.all(np.abs(y - x) <= s / 2)
        a = np.abs(x).reshape(1, 3, 4, -1).max(-1)
        assert np.all(s[:, :, ::16, 0] <= a / 64) and np.all(s[:, :, ::16, 0] > a / 128)
        assert np.array_equal(q4_ref.bf16(y.astype(np.float32)), y)         # exact in bf16
    assert ref.scale_of(1.0) == 2.0 ** -6 and ref.scale_of(1.99) == 2.0 ** -6 and ref.scale_of(2.0 ** -130) == 2.0 ** -126
    # rows one by one, in any order of sizes, give what they give at once
    row = {t: q4_ref.bf16(rng.standard_normal(128) * 4.0 ** rng.integers(-3, 4)) for t in range(16)}
    at_once, one_by_one = np.zeros(16416, np.uint8), np.zeros(16416, np.uint8)
    ref.put(at_once, 1, row, [], True)
    for t in range(16):
        ref.put(one_by_one, 1, {t: row[t]}, list(range(t)), True)
    assert np.array_equal(at_once, one_by_one)
