"""Barriers between CTAs that share memory order it: an arrival releases and a wait acquires, in every kernel."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitwise_aligned_causal_gb300", "csrc")


def test_no_barrier_is_relaxed():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for op in re.findall(r"(?:mbarrier\.(?:arrive|try_wait|test_wait)|barrier\.cluster\.(?:arrive|wait))[\w.:]*", open(path).read()):
            seen += 1
            assert "relaxed" not in op, (os.path.basename(path), op)
    assert seen > 5
