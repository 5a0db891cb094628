"""What the library launches, seen by a CUDA runtime that runs nothing."""
import json

import pytest

import fake_cuda


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from sparse_paged_kv_score_gb300 import build
    build.build()
    return fake_cuda.build(str(tmp_path_factory.mktemp("fake")))


ATTEND = """
import json, re
got = []
for sms in {sms}:
    f.rt.fake_sms(sms)
    for Hk in (1, 8):
        h = f.handle(True, Hk)
        f.events()
        for B in {batches}:
            for n in {lists}:
                for G in (1, 5, 16):
                    assert f.lib.sparse_decode_attn(h, 4096, B, G * Hk, 4096, 9, 4096, 4096, n, 4096, 4096, 4096, None) == 0
                    (e,) = f.events()
                    mode, grid, parts = map(int, re.fullmatch(
                        r"launch \\S*attn_q4_kernel\\S*ModeE(\\d)\\S* (\\d+) parts (\\d+)", e).groups())
                    got.append([sms, B * Hk, n, mode, grid, parts])
print(json.dumps(got))
"""


@pytest.mark.parametrize("sms", [[152, 148], [90, 86, 85], [64, 40], [20, 8, 1]])
def test_every_part_of_a_unit_has_its_cta(fake, sms):
    """4-bit attention: where CTAs take parts of units (mode 2), or may take them as the lists turn out (mode 1), the
    grid has a CTA for every part of every unit, on a device or a share of one with few SMs as well."""
    program = ATTEND.format(sms=sms, batches=[1, 2, 7, 13, 31, 32, 61, 100, 200, 256, 300, 500],
                            lists=[1, 3, 4, 5, 16, 17, 33, 65, 129, 700])
    seen = set()
    for m, U, n, mode, grid, parts in json.loads(fake_cuda.run(fake, program)):
        assert 1 <= grid <= 3 * m and parts >= 1, (m, U, n, mode)
        if mode == 2:
            assert grid == U * parts, (m, U, n)
        if mode == 1:
            assert grid >= U * parts, (m, U, n)
        seen.add(mode)
    assert seen == {0, 1, 2}


def test_a_bf16_handle_prepares_no_4bit_kernel(fake):
    """Creating a handle loads the kernels that its own calls launch, not the other format's, a later one's too."""
    program = """
import json
a, b, c = [f.handle(q4, 2) and f.events() for q4 in (False, True, False)]
print(json.dumps([a, b, c]))
"""
    bf16, q4, again = json.loads(fake_cuda.run(fake, program))
    sets = [{e.split()[1] for e in x if e.startswith("set ")} for x in (bf16, q4, again)]
    assert not any("attn_q4" in name for name in sets[0] | sets[2])
    assert len([name for name in sets[1] if "attn_q4" in name]) == 9 and not any("prefill" in name for name in sets[1])
    assert sets[0] == sets[2] and "?" not in sets[0] | sets[1]


def test_calls_for_bf16_pools_refuse_a_4bit_handle(fake):
    """Every entry point that reads or writes bf16 pages: SPKV_EUNSUPPORTED on a 4-bit handle, nothing launched;
    the same arguments pass on a bf16 handle (where a host pool that is not pinned ends the retrieval)."""
    program = """
import ctypes, json
P = 4096
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
)
got = {}
for name, args in calls.items():
    got[name] = []
    for q4 in (True, False):
        h = f.handle(q4, 2)
        f.events()
        status = getattr(f.lib, name)(h, *args)
        got[name].append([status, len(f.events())])
name = "lazy_rope_decode_attn_docs"
got[name] = []
for h in (f.handle(True, 2), h):    # the last: the plan's
    f.events()
    status = f.lib.lazy_rope_decode_attn_docs(h, plan, P, P, P, P, P, 1e4, P, P, None)
    got[name].append([status, len(f.events())])
print(json.dumps(got))
"""
    got = json.loads(fake_cuda.run(fake, program))
    assert len(got) == 12
    for name, (q4, bf16) in got.items():
        assert q4 == [-6, 0], name
        if name.startswith("retrieve"):
            assert bf16 == [-1, 0], name
        else:
            assert bf16[0] == 0 and bf16[1] >= (name != "lazy_docs_plan_create"), (name, bf16)
