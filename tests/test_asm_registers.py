"""Inline assembly names every register that it writes: m0, which no operand stands for, as an output or a clobber."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(p for end in ("hip", "hpp")
                 for p in glob.glob(os.path.join(ROOT, "ggml_iq_codebook_imatrix_amd", "*", "*." + end)))


def statements(text):
    """The asm statements of a source, from the keyword to the parenthesis that closes it."""
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_m0_is_named_where_it_is_written(path):
    for s in statements(open(path).read()):
        if re.search(r"\bs_\w+ m0\b", s):
            assert re.search(r'"=&?\{m0\}"|"m0"', s), s
