"""Inline assembly of the kernels tells the compiler every register it writes."""
import os
import re

import pytest

from sparse_moe_layer_03_amd import build


def statements(text):
    """Source text of every asm statement, up to its closing parenthesis (parentheses in strings do not count)."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, quoted, i = 1, False, m.end()
        while depth:
            c = text[i]
            if c == "\\" and quoted:
                i += 1
            elif c == '"':
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


def writes_m0(statement):
    return re.search(r"\bs_mov_b32 m0\b", statement) is not None


def names_m0(statement):
    return re.search(r':[^:]*"m0"[^:]*\)$', statement, re.S) is not None


def test_rule_sees_a_missing_clobber():
    load = 'asm volatile("s_mov_b32 m0, %0\\n\\tglobal_load_lds_dword %1, off" ::"s"(a), "v"(b) : "memory"'
    (bad,), (good,) = statements(load + ");"), statements(load + ', "m0");')
    assert writes_m0(bad) and not names_m0(bad) and names_m0(good)


@pytest.mark.parametrize("source", [os.path.basename(s) for s in build.sources()])
def test_m0_is_named(source):
    with open(os.path.join(build.CSRC, source)) as f:
        for s in statements(f.read()):
            assert not writes_m0(s) or names_m0(s), s
