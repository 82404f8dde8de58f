"""Inline assembly in the kernels names every register that it writes itself."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "state_space_recurrence_amd", "csrc")


def _statements(text):
    """The operands of each asm statement, from its opening to its closing parenthesis."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, quoted, i = 1, False, m.end()
        while depth:
            ch = text[i]
            if ch == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (ch == "(") - (ch == ")")
            i += 1
        yield text[m.end():i - 1]


def undeclared(statement):
    """Physical registers that a statement's instructions write and its clobbers do not name."""
    parts, quoted, cut = [], False, 0
    for i, ch in enumerate(statement):
        if ch == '"':
            quoted = not quoted
        elif ch == ":" and not quoted:
            parts.append(statement[cut:i])
            cut = i + 1
    parts.append(statement[cut:])
    code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', parts[0]))
    clobbers = set(re.findall(r'"([^"]*)"', parts[3])) if len(parts) > 3 else set()
    written = set()
    for ins in re.split(r"\\n(?:\\t)?", code):
        m = re.match(r"\s*\S+\s+(m0|vcc|exec|scc|[sv]\d+)\b", ins)
        if m:
            written.add(m.group(1))
    return written - clobbers


def test_reader_of_asm_statements():
    text = r'asm volatile("s_mov_b32 m0, %1\n\ts_nop 0" ::"v"(f(x)), "s"(y) : "memory"); asm volatile("" : "+v"(a), "+v"(b));'
    first, second = _statements(text)
    assert undeclared(first) == {"m0"} and undeclared(second) == set()
    assert undeclared(first.replace('"memory"', '"m0", "memory"')) == set()


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))),
                         ids=os.path.basename)
def test_registers_written_are_declared(path):
    with open(path) as f:
        for s in _statements(f.read()):
            assert not undeclared(s), s
