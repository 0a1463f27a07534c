"""Bounded waits in the kernels' sources (no GPU needed).

Each lane of a warp reads the timer for itself, so near the limit some lanes of a per-lane wait may give up while others see the
copy land.  What follows a wait are products and shuffles of all lanes, which a part of a warp must not enter: there the
whole warp has to decide (mbar_wait_warp, or a vote over the single tests).  A per-lane wait serves only where nothing
depends on its answer: the last copies in flight, before a warp leaves.
"""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "paged_kv_gqa_block_gb300")
SOURCES = sorted(f for d in ("csrc", "serving") for f in glob.glob(os.path.join(PKG, d, "*.cu*")))


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def test_no_branch_depends_on_a_wait_of_one_lane():
    waits = 0
    for path in SOURCES:
        text = code(path)
        for m in re.finditer(r"\bmbar_wait\s*\(", text):
            before = text[:m.start()].rstrip()
            if os.path.basename(path) == "pda_ptx.cuh" and before.endswith("bool"):
                continue                                     # its definition
            waits += 1
            assert before.endswith("(void)"), f"{os.path.basename(path)}: {text[m.start() - 40:m.end() + 60]!r}"
    assert waits > 0


def test_single_tests_of_a_phase_are_voted_on():
    for path in SOURCES:
        text = code(path)
        if os.path.basename(path) == "pda_ptx.cuh":
            text = text[text.index("mbar_wait_warp"):]       # the wrappers themselves and the per-lane form stand before it
        for m in re.finditer(r"\bmbar_(try|test)_wait\s*\(", text):
            start = max(text.rfind(";", 0, m.start()), text.rfind("{", 0, m.start()), text.rfind("}", 0, m.start()))
            statement = text[start:text.index(";", m.end())]
            following = text[m.end():m.end() + 400]
            voted = "__all_sync" in statement or re.search(r"bool ok = [^;]*$", text[start:m.start()]) and "__all_sync" in following
            assert voted, f"{os.path.basename(path)}: {statement!r}"


def test_the_vote_is_of_the_answer_and_of_the_limit():
    text = code(os.path.join(PKG, "csrc", "pda_ptx.cuh"))
    body = text[text.index("bool mbar_wait_warp"):]
    body = body[:body.index("\n}\n")]
    assert len(re.findall(r"if \(__all_sync\([^;]*\) return true;", body)) == 2
    assert re.search(r"if \(__any_sync\([^;]*limit_ns\)\) return false;", body)
    assert body.count("return") == 3
