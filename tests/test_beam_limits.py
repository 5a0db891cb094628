"""What spkv.h says of beam_select in numbers, against the tests' own bound and the library."""
import math
import os
import re

import beam_ref as ref

HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "spkv.h")).read()


def test_the_documented_error_of_a_beams_sum():
    """The bound that spkv.h gives for a beam's log of the sum of exponentials is what its sums are derived to keep."""
    text = " ".join(line.strip(" *") for line in HEADER.split("\n"))
    a, b, c = map(float, re.search(r"off by at most \((\S+) ln\(V \+ 1\) \+ (\d+) \+ V / (\d+)\) 2\^-23", text).groups())
    for V in [1, 2, 1023, 1024, 1025, 32000, 32768, 32769, 128256, 1 << 20, 1 << 24]:
        stated = (a * math.log(V + 1) + b + V / c) * 2.0 ** -23
        assert ref.lse_error(V) <= stated <= 1.05 * ref.lse_error(V) + 2.0 ** -23
