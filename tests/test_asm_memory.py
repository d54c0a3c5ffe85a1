"""Inline assembly that reads or writes memory, or waits, is volatile, so that the compiler keeps such
statements in order, and loads of global memory say that they read it, on the CPU: without, a load is
arithmetic on its address, which may be moved before the wait for what it reads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_65_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))
# what may stand without: moves and arithmetic between registers
PLAIN = re.compile(r"^(\.reg|mov|add|sub|mul|fma|max|min|ex2|setp|selp|and|elect)\b")


def statements(text):
    """(the words after asm, its instructions, the rest of its operands) of each asm statement."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"\basm\b([^(]*)\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if quoted:
                at += c == "\\"
                quoted = c != '"'
            else:
                quoted = c == '"'
                depth += (c == "(") - (c == ")")
            at += 1
        body = text[m.end():at - 1]
        code = re.match(r'(\s*"(?:[^"\\]|\\.)*")+', body)
        words = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', code.group(0)))
        words = re.sub(r"\\[nt]", " ", words)
        yield m.group(1).strip(), words, body[code.end():]


def test_statements_are_found():
    got = list(statements('x; asm("add.f32 %0, (a);" : "=f"(y)); asm volatile("ld" ".x [%1];" ::: "memory");'))
    assert [g[:2] for g in got] == [("", "add.f32 %0, (a);"), ("volatile", "ld.x [%1];")]
    assert sum(len(list(statements(open(os.path.join(CSRC, f)).read()))) for f in SOURCES) > 50


@pytest.mark.parametrize("name", SOURCES)
def test_loads_are_volatile(name):
    with open(os.path.join(CSRC, name)) as f:
        for how, code, operands in statements(f.read()):
            parts = [p.strip().lstrip("{").strip() for p in re.split(r";", code)]
            if all(PLAIN.match(re.sub(r"^@\w+\s+", "", p)) for p in parts if p.strip("{} ")):
                continue
            assert "volatile" in how, (name, code)
            if "ld.global" in code or "griddepcontrol.wait" in code:
                assert '"memory"' in operands, (name, code)
