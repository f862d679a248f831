"""CPU tests of the kernels' source text."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_10_amd", "csrc")
SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".h", ".hip", ".cpp")))


def asm_statements(name):
    """(instructions, whole text) of each inline assembly statement of a source file."""
    src = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
    for m in re.finditer(r"__asm__\s*(?:volatile\s*)?\(", src):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = src[at]
            quoted ^= c == '"' and src[at - 1] != "\\"
            depth += 0 if quoted else (c == "(") - (c == ")")
            at += 1
        text = src[m.end():at - 1]
        template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split(":")[0]))
        yield [x.split()[0] for x in re.split(r"\\n\\t|\\n|;", template) if x.split()], text


@pytest.mark.parametrize("name", SOURCES)
def test_inline_assembly_computes_nothing(name):
    """Copies to LDS, waits and barriers only. A vector instruction in inline assembly could read a matrix
    product's result too early: the compiler leaves the wait states only before instructions that it knows."""
    for ops, text in asm_statements(name):
        for op in ops:
            assert re.fullmatch(r"s_mov_b32|s_nop|s_waitcnt|s_barrier|global_load_lds_dword(x4)?", op), text


@pytest.mark.parametrize("name", SOURCES)
def test_inline_assembly_names_what_it_writes(name):
    """M0 is written by the copies to LDS: as a clobber, so that nothing is held there across them."""
    for ops, text in asm_statements(name):
        if re.search(r"s_mov_b32 m0", text):
            assert re.search(r'"m0"', text.split(":")[-1]), text


@pytest.mark.parametrize("name", SOURCES)
def test_copies_wait_for_their_base(name):
    """A memory instruction may read a scalar base five wait states after a vector instruction wrote it (a
    readfirstlane, or a spilled register's return); in inline assembly the compiler leaves none of them."""
    for ops, text in asm_statements(name):
        if any(op.startswith("global_load") for op in ops) and not re.search(r"global_load\w+ %\d+, off", text):
            before = text[:text.index("global_load")]
            states = sum(int(n) + 1 for n in re.findall(r"s_nop (\d+)", before)) + len(re.findall(r"s_mov_b32", before))
            assert states >= 5, text
