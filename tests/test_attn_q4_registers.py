"""What the compiler makes of the 4-bit attention's kernels, whose warps keep a softmax's state in registers."""
import os
import re
import subprocess

from sparse_paged_kv_score_gb300 import build


def test_kernels_of_one_warp_a_page_spill_nothing(tmp_path):
    """Up to 8 query heads a kv head.  (With 9 to 16 two warps share a page, and two of the three instances load 16 and 28 bytes.)"""
    source = os.path.join(build.CSRC, "attn_q4.cu")
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas", "-v", "-c", source, "-o",
                        str(tmp_path / "attn_q4.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function properties for \S*attn_q4_kernelILi(\d)E\S*ModeE(\d)\S*\n\s*\d+ bytes stack frame, (\d+) bytes spill stores, "
                       r"(\d+) bytes spill loads", r.stderr)
    assert len(found) == 9
    for groups, mode, stores, loads in found:
        assert (int(stores), int(loads)) <= ((0, 0) if groups == "1" else (16, 28)), (groups, mode, stores, loads)
