"""Rules of the instructions that the kernels hold as text, which the compiler does not look into."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_qmm_gemv_amd", "csrc")


def statements():
    """(place, instructions, everything between the parentheses) of every asm statement."""
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
            depth, at, quoted = 1, m.end(), False
            while depth:
                c = text[at]
                if c == '"' and text[at - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += {"(": 1, ")": -1}.get(c, 0)
                at += 1
            body = text[m.end():at - 1]
            template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', re.split(r"(?<!:):(?!:)", re.sub(r'"(?:[^"\\]|\\.)*"',
                               lambda q: q.group().replace(":", "\0"), body))[0])).replace("\0", ":")
            lines = [x.strip() for x in template.replace("\\n", "\n").replace("\\t", " ").split("\n")]
            yield "%s:%d" % (name, text.count("\n", 0, m.start()) + 1), [x for x in lines if x], body


ALL = list(statements())


def test_there_are_statements():
    assert len(ALL) >= 8 and sum("lds" in " ".join(x) for _, x, _ in ALL) >= 4


@pytest.mark.parametrize("place,lines,body", ALL, ids=[p for p, _, _ in ALL])
def test_a_written_m0_is_named(place, lines, body):
    if any(re.match(r"s_\w+\s+m0\b", x) for x in lines):
        assert re.search(r':[^:]*"m0"[^:]*$', body), place


@pytest.mark.parametrize("place,lines,body", ALL, ids=[p for p, _, _ in ALL])
def test_memory_instructions_wait_for_scalar_operands(place, lines, body):
    # Five wait states lie between a vector instruction's write of a scalar register and a memory instruction's read of it;
    # within a statement its own instructions have to make them up (an instruction is one, s_nop n is n + 1).
    if not re.search(r'"s"\s*\(', body):
        return
    states = 0
    for x in lines:
        if re.match(r"(buffer|global|flat)_", x):
            assert states >= 5, place
        nop = re.match(r"s_nop\s+(\d+)", x)
        states += int(nop[1]) + 1 if nop else 1
