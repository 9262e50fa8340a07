"""The kernels' checks of a sequence's start and row count, which come from device memory and may be anything: taken out
of the sources and worked out in 32-bit arithmetic that wraps, against whole numbers."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitwise_aligned_causal_gb300", "csrc")
NAME = r"(\w+(?:\.\w+)?)"
REFUSED = re.compile(rf"{NAME} < 0 \|\| {NAME} < 0 \|\| \2 > ([\w.]+) \|\| ([^|()]+?) ?(?:\)|\|\|)")
ACCEPTED = re.compile(rf"{NAME} >= 0 && {NAME} >= [01] && \2 <= ([\w.]+) && ([^&();]+);")
KERNELS = ("kb_append.cu", "kb_cache8.cu", "kb_decode.cu", "kb_decode8.cu", "kb_prefill2.cu", "kb_select.cu", "kb_sparse.cuh",
           "kb_weights.cu", "kb_weights_rows.cu")


class Int32(int):
    def __add__(self, o):
        return Int32((int(self) + int(o) + 2 ** 31) % 2 ** 32 - 2 ** 31)

    def __sub__(self, o):
        return Int32((int(self) - int(o) + 2 ** 31) % 2 ** 32 - 2 ** 31)


def checks(path):
    """(refuses?, name of the start, of the row count, last comparison) of every check in a file."""
    text = re.sub(r"\s+", " ", open(path).read())
    return [(refused, m[1], m[2], m[4]) for refused, rule in ((True, REFUSED), (False, ACCEPTED)) for m in rule.finditer(text)]


def in_cache(check, start, rows, cap):
    refused, s, n, last = check
    names = {s: Int32(start), n: Int32(rows)}
    terms = re.sub(NAME, lambda m: f"names[{m[1]!r}]" if m[1] in names else "cap", last)
    return eval(terms, {"names": names, "cap": Int32(cap)}) != refused


def test_every_kernel_that_reads_starts_has_one():
    found = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*")) if checks(p)}
    assert found == set(KERNELS)


@pytest.mark.parametrize("name", KERNELS)
def test_no_start_passes_that_lies_outside(name):
    cap = 1024
    for check in checks(os.path.join(CSRC, name)):
        for rows in (0, 1, 2, 31, 300, 1024):                    # (0 <= rows <= the call's rows by the comparisons before)
            for start in (0, 1, cap - rows - 1, cap - rows, cap - rows + 1, cap, cap + 1, 2 ** 31 - rows - 1, 2 ** 31 - rows, 2 ** 31 - 2,
                          2 ** 31 - 1):
                if 0 <= start < 2 ** 31:
                    assert in_cache(check, start, rows, cap) == (start + rows <= cap), (check, start, rows)
