"""Arrays in static shared memory that a kernel reads or writes in words wider than their elements are declared as aligned as
those words: a faulting address otherwise hangs on where the compiler places its neighbours."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitwise_aligned_causal_gb300", "csrc")

# file, array, bytes of the widest word
WIDE = [("kb_evict.cu", "hist", 8),                      # pairs of bins, from the cluster's CTAs
        ("kb_segment.cu", "held", 16)]                   # partials, by cp.async and as four floats


@pytest.mark.parametrize("name,array,word", WIDE)
def test_wide_words_are_aligned(name, array, word):
    text = open(os.path.join(CSRC, name)).read()
    m = re.search(rf"__shared__ ([^;\[]*)\b{array}\[", text)
    assert m, f"{array} is not a static shared array of {name}"
    aligned = re.search(r"__align__\((\d+)\)", m[1])
    assert aligned and int(aligned[1]) >= word, m[0]
