"""The kernels' asm statements (no GPU): what they overwrite, they declare."""

import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "fully_sharded_amd", "csrc", "*")))


def statements(text):
    """Every asm statement, up to its closing bracket."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text[m.end():at - 1]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_special_registers_are_declared(path):
    """A statement that writes M0, VCC or EXEC names it among its outputs or
    clobbers, or the compiler may keep a value of its own there across it."""
    with open(path) as f:
        for body in statements(f.read()):
            parts = body.split(":")
            for reg in ("m0", "vcc", "exec"):
                if re.search(rf"\b[sv]_\w+ {reg}\b", parts[0]):
                    assert len(parts) > 1 and f"{{{reg}}}" in parts[1] or \
                        len(parts) > 3 and f'"{reg}"' in parts[-1], body


def test_statements_are_found():
    got = list(statements('asm volatile("s_mov_b32 m0, %0" ::"s"(f(1)) : "memory"); asm("" ::: );'))
    assert got == ['"s_mov_b32 m0, %0" ::"s"(f(1)) : "memory"', '"" ::: ']
