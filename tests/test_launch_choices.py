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
