"""What the 4-bit cache and the rotating append refuse on the host, before any CUDA call."""
import ctypes
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from sparse_paged_kv_score_gb300 import build
    build.build()
    from sparse_paged_kv_score_gb300 import _abi
    return _abi.load()


# n_kv_heads, head_dim, page_tokens, subblock, n_phys_pages, kv_pool, k_scale, v_scale, ksum, page_cnt, max_units, ksum_bf16
GOOD = dict(n_kv_heads=2, head_dim=128, page_tokens=64, subblock=16, n_phys_pages=4, kv_pool=4096, k_scale=4096, v_scale=4096,
            ksum=4096, page_cnt=4096, max_units=0, ksum_bf16=0)


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=64), "EUNSUPPORTED"), (dict(page_tokens=32), "EUNSUPPORTED"), (dict(subblock=8), "EUNSUPPORTED"),
    (dict(n_kv_heads=0), "EINVAL"), (dict(n_kv_heads=-1), "EINVAL"), (dict(n_phys_pages=0), "EINVAL"),
    (dict(kv_pool=None), "EINVAL"), (dict(kv_pool=4104), "EINVAL"), (dict(k_scale=None), "EINVAL"),
    (dict(v_scale=None), "EINVAL"), (dict(page_cnt=None), "EINVAL"), (dict(ksum=4104), "EINVAL"),
    (dict(max_units=-1), "EINVAL"), (dict(max_units=4097), "EINVAL"), (dict(ksum_bf16=2), "EINVAL"),
    (dict(n_phys_pages=1 << 30), "EUNSUPPORTED"), (dict(n_phys_pages=(1 << 31) - 1, n_kv_heads=4), "EUNSUPPORTED")])
def test_descriptions(lib, bad, status):
    from sparse_paged_kv_score_gb300 import _abi
    out = ctypes.c_void_p(1)
    d = _abi.SpkvDescQ4(**{**GOOD, **bad})
    assert lib.paged_kv_create_q4(ctypes.byref(d), None, ctypes.byref(out)) == getattr(_abi, "SPKV_" + status)
    assert not out.value
    assert lib.paged_kv_create_q4(None, None, ctypes.byref(out)) == _abi.SPKV_EINVAL
    assert lib.paged_kv_create_q4(ctypes.byref(d), None, None) == _abi.SPKV_EINVAL


def test_no_handle(lib):
    from sparse_paged_kv_score_gb300 import _abi
    assert lib.paged_kv_append_rope(None, 16, 256, 16, 256, 1, 1, None, 16, 16, 1, None, None, 0, 0, None, None) == _abi.SPKV_EINVAL
    assert lib.paged_kv_unpack_q4(None, 16, 1, 16, 16, None) == _abi.SPKV_EINVAL


def test_cache_arguments():
    import sparse_paged_kv_score_gb300 as spkv
    pool = torch.zeros(2, 3, 9216, dtype=torch.uint8)
    g = torch.ones(2)
    with pytest.raises(ValueError, match="9216"):
        spkv.paged_kv_create_q4(pool[0], g, g, None, None)
    with pytest.raises(ValueError, match="page_cnt"):
        spkv.paged_kv_create_q4(pool, g, g, torch.zeros(2, 3, 4, 128), None)
    with pytest.raises((ValueError, TypeError)):
        spkv.paged_kv_create_q4(pool, g, g, None, None)   # not on a GPU


def test_append_and_unpack_arguments():
    import sparse_paged_kv_score_gb300 as spkv
    cache = SimpleNamespace(n_kv_heads=2, handle=None, tensors=[torch.zeros(1)])
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    L, pt = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        spkv.paged_kv_append_rope(cache, k, k, L, pt)
    with pytest.raises(TypeError, match="bfloat16"):
        spkv.paged_kv_append_rope(cache, k.float(), k, L, pt)
    with pytest.raises(ValueError, match="CUDA"):
        spkv.paged_kv_append_rope(cache, k.to("meta"), k, L, pt)
    with pytest.raises((TypeError, ValueError)):
        spkv.paged_kv_unpack_q4(cache, L, k, k)
