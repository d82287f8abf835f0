"""An instruction in which the lanes of a warp meet is not a function of its
operands alone: written as a plain asm, the compiler may move it into a branch
that only some of the lanes take.  Each is volatile.  Read from the sources."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bmmc_index_transforms_gb300", "csrc")


def test_instructions_in_which_lanes_meet_are_volatile():
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\b\s*(volatile\b)?\s*\((.*?)\"\s*(?::|\))", code, re.S):
            if re.search(r"\.sync\b|\bbar(rier)?\.|\bvote\.|\bmatch\.|\belect\.", m.group(2)):
                seen += 1
                assert m.group(1), f"{name}: {' '.join(m.group(2).split())}"
    assert seen
