"""Inline assembly in the kernels declares the special registers it writes."""

from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "row_radix_top_amd", "csrc")
SPECIAL = {"m0": r"m0", "vcc": r"vcc(?:_lo|_hi)?", "exec": r"exec(?:_lo|_hi)?"}


def _statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
            end, depth, quoted = m.end(), 1, False
            while depth:
                c = text[end]
                quoted ^= c == '"' and text[end - 1] != "\\"
                depth += 0 if quoted else {"(": 1, ")": -1}.get(c, 0)
                end += 1
            yield os.path.basename(path), text[m.end():end - 1]


def test_there_are_some():
    assert any("m0" in s for _, s in _statements())


@pytest.mark.parametrize("register", SPECIAL)
def test_special_registers_that_are_written_are_clobbered(register):
    for name, s in _statements():
        code = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)*)', s).group(1)
        lines = re.split(r'\\n|\\t|"|\n', code)
        if any(re.match(rf"\s*\w+\s+{SPECIAL[register]}\s*,", line) for line in lines):
            assert f'"{register}"' in s[len(code):], f"{name}: {s}"
