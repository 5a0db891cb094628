"""The ncu summaries under profiles/more_operators/ each give the commands that produced them: a case of
perf/more_operators.py, one launch of one of the library's kernels, the clocks left alone."""
import glob
import os
import re
import shlex

import perf.more_operators as operators

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUMMARIES = sorted(glob.glob(os.path.join(ROOT, "profiles", "more_operators", "*.md")))


def test_every_capture_can_be_repeated():
    kernels = "".join(open(p).read() for p in glob.glob(os.path.join(ROOT, "sparse_paged_kv_score_gb300", "csrc", "*.cu")))
    names = {c["name"] for c in operators.listed()}
    assert SUMMARIES
    for path in SUMMARIES:
        text, n = open(path).read(), 0
        for block in re.findall(r"```\n(.*?)```", text, re.S):
            cmd = shlex.split(block.replace("\\\n", ""))
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
    """Template arguments of the attention's instances as the source has them: query heads at most, mode."""
    source = open(os.path.join(ROOT, "sparse_paged_kv_score_gb300", "csrc", "attn_q8.cu")).read()
    modes = re.search(r"enum Mode \{(.*?)\}", source)[1].replace(" ", "").split(",")
    heads = re.findall(r"struct Shape8<(\d+)>", source)
    for path in SUMMARIES:
        for args in re.findall(r"attn_q8_kernel<(.*?)>", open(path).read(), re.S):
            h, mode = (a.strip() for a in args.split(","))
            assert h in heads and mode in modes, (path, args)


def test_cases_have_two_of_each_operator():
    """Of each kind of case several are listed, drawn ones are of the same kinds, and what a pass must move is known."""
    import collections
    import random
    kinds = collections.Counter(c["kind"] for c in operators.listed())
    assert set(kinds) == {"chunk", "unpack", "attend", "step", "select", "reorder"} and 4 <= sum(kinds.values()) <= 12
    assert all(n >= 2 for k, n in kinds.items() if k != "step")     # a step is an append and an attention
    rng = random.Random(0)
    drawn = [operators.draw(rng) for _ in range(300)]
    assert {c["kind"] for c in drawn} == set(kinds)
    assert all(operators.work(c)["bytes"] > 0 for c in drawn + operators.listed())
