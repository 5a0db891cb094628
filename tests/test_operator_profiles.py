"""The ncu summaries under profiles/operators/ each give the commands that produced them: a case of perf/operators.py,
one launch of one of the library's kernels, the clocks left alone."""
import glob
import os
import re
import shlex

import perf.operators as operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUMMARIES = sorted(glob.glob(os.path.join(ROOT, "profiles", "operators", "*.md")))


def _commands(path):
    for block in re.findall(r"```\n(.*?)```", open(path).read(), re.S):
        yield shlex.split(block.replace("\\\n", ""))


def test_every_capture_can_be_repeated():
    kernels = "".join(open(p).read() for p in glob.glob(os.path.join(ROOT, "sparse_paged_kv_score_gb300", "csrc", "*.cu")))
    names = {c["name"] for c in operators.listed()}
    assert SUMMARIES
    for path in SUMMARIES:
        text, n = open(path).read(), 0
        for cmd in _commands(path):
            assert cmd[0] == "ncu" and cmd[cmd.index("--clock-control") + 1] == "none", path
            assert cmd[cmd.index("-c") + 1] == "1", path
            kernel = cmd[cmd.index("-k") + 1].removeprefix("regex:")
            assert re.search(rf"\b{kernel}\w*\(", kernels) and f"`{kernel}" in text, path
            program = cmd[cmd.index("python") + 2]
            compile(program, path, "exec")
            assert re.search(r"c\['name'\] == '(.*?)'", program)[1] in names, path
            n += 1
        assert n == text.count("| `gpu__time_duration.sum` |") > 0, path    # one for each table


def test_captures_name_the_kernels_that_are_there():
    """Template arguments of the attention's instances as the source has them: head groups a page, packing, mode."""
    source = open(os.path.join(ROOT, "sparse_paged_kv_score_gb300", "csrc", "attn_q4.cu")).read()
    modes = re.search(r"enum Mode \{(.*?)\}", source)[1].replace(" ", "").split(",")
    for path in SUMMARIES:
        for args in re.findall(r"attn_q4_kernel<(.*?)>", open(path).read(), re.S):
            groups, pack, mode = (a.strip() for a in args.replace("\n", " ").split(","))
            assert groups in ("1", "2") and pack in ("true", "false") and mode in modes, (path, args)
