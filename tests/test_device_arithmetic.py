"""CPU tests of the kernels' source text: the smaller and the larger of two numbers of different types.

HIP's max and min of an int and an unsigned (a count of bits is one) are those of two doubles: from a count of none, less
one, they make 4294967295.0, and an index of it."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_10_amd", "csrc")
SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".h", ".hip", ".cpp")))


def calls(src, name):
    """The texts between the parentheses of calls of a function."""
    for m in re.finditer(r"\b%s\(" % name, src):
        depth, at = 1, m.end()
        while depth:
            depth += (src[at] == "(") - (src[at] == ")")
            at += 1
        yield src[m.end():at - 1]


@pytest.mark.parametrize("name", SOURCES)
def test_counts_of_bits_are_compared_as_integers(name):
    src = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
    for f in ("max", "min"):
        for args in calls(src, f):
            for count in re.finditer(r"__popc(ll)?\(|__clz(ll)?\(", args):
                assert re.search(r"static_cast<int(32_t|64_t)?>\($", args[:count.start()]), f"{f}({args})"
