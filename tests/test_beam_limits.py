"""What spkv.h says of beam_select in numbers, against the tests' own bound and the library."""
import json
import math
import os
import re

import pytest

import beam_ref as ref
import fake_cuda
from sparse_paged_kv_score_gb300 import build

HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "spkv.h")).read()


def test_the_documented_error_of_a_beams_sum():
    """The bound that spkv.h gives for a beam's log of the sum of exponentials is what its sums are derived to keep."""
    text = " ".join(line.strip(" *") for line in HEADER.split("\n"))
    a, b, c = map(float, re.search(r"off by at most \((\S+) ln\(V \+ 1\) \+ (\d+) \+ V / (\d+)\) 2\^-23", text).groups())
    for V in [1, 2, 1023, 1024, 1025, 32000, 32768, 32769, 128256, 1 << 20, 1 << 24]:
        stated = (a * math.log(V + 1) + b + V / c) * 2.0 ** -23
        assert ref.lse_error(V) <= stated <= 1.05 * ref.lse_error(V) + 2.0 ** -23


@pytest.mark.parametrize("kind,size", [(0, 4), (1, 2), (2, 2)])
def test_the_largest_calls_of_a_request(tmp_path, kind, size):
    """W rows, each rounded up to 4096 bytes, of 2^27 bytes together are taken, one group of 4096 more is refused before
    anything is launched (9 x 3641 groups are one too many), be the rows' bytes as they are fewer than that too."""
    build.build()
    a = 4096 // size          # elements of a group
    cases = [(64, 512 * a, 0), (64, 512 * a + 1, -6), (2, 8192 * a, 0), (63, 520 * a, 0), (63, 520 * a + 5, -6),
             (9, 3640 * a, 0), (9, 3640 * a + 1, -6)]
    program = f"""
import ctypes, json
P = 4096
h = f.handle(False, 2, max_units=64)
got = []
for W, V, _ in {cases!r}:
    plan = ctypes.c_void_p()
    assert f.lib.beam_plan_create(h, W, V, ctypes.byref(plan)) == 0
    f.events()
    got.append([f.lib.beam_select(h, plan, P, {kind}, V, 1, W, V, P, 8, P, P, P, None), len(f.events())])
    f.lib.beam_plan_destroy(plan)
print(json.dumps(got))
"""
    got = json.loads(fake_cuda.run(fake_cuda.build(str(tmp_path)), program))
    assert got == [[status, 0 if status else 2] for _, _, status in cases]
    for W, V, status in cases:
        assert (W * -(-V * size // 4096) * 4096 <= 2 ** 27) == (status == 0)
    assert 63 * (520 * a + 5) * size <= 2 ** 27      # (the rows as they are)
