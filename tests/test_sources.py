"""What the kernels' sources may not hold: checked on the text alone, without a GPU."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_means_clustering_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip")))


def statements(text):
    """The instructions' text of each asm statement (its string literals before the first colon, joined)."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"\basm\b\s*(?:volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", text):
        yield "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m[1]))


def instructions(asm):
    return [i.strip() for i in re.split(r"\\n|\\t|;", asm) if i.strip()]


def test_the_check_sees_instructions():
    assert [instructions(s) for s in statements('x; asm volatile("v_a %0\\n\\t" "v_b %0" : "+v"(x)); asm("" : "+s"(y)); // asm("c")')] == [
        ["v_a %0", "v_b %0"], []]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_an_asm_statement_holds_one_instruction(path):
    """A vector instruction that reads what the one before it wrote (the carry of a comparison, a lane exchange's source)
    may need wait states between the two.  The compiler knows them and fills them in, but not inside a statement."""
    with open(path) as f:
        for asm in statements(f.read()):
            assert len(instructions(asm)) <= 1, asm
