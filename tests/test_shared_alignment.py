"""Byte arrays in shared memory that kernels also access by wider words state
their alignment: without it a byte array may start anywhere."""

import os
import re

import pytest

from tests.test_kernel_sources import SOURCES


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_byte_arrays_state_their_alignment(path):
    with open(path) as f:
        text = re.sub(r"//.*", "", f.read())
    for decl, name in re.findall(r"(?<!extern )(__shared__[^;\[]*\b(?:u?int8_t|char)\s+(\w+)\s*\[)", text):
        wide = re.search(r"reinterpret_cast<[^>]*(?:u?int(?:16|32|64)_t|u?int[24]|float\w*)\s*\*>\(&" + name + r"\b", text)
        assert not wide or re.search(r"__align__\((?:4|8|16)\)|alignas\((?:4|8|16)\)", decl), decl
