"""Inline assembly of the kernels, read as text: what it uses is named to the
compiler."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_q4g128_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
            depth, at = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
            yield os.path.basename(path), " ".join(text[m.start():at].split())


def test_m0_is_an_operand():
    """Loads to LDS take their address from m0: the compiler writes it (an
    operand in m0), and no statement writes it behind its back."""
    loads = [(f, s) for f, s in statements() if re.search(r"\blds\b", s)]
    assert loads
    for f, s in loads:
        assert '"{m0}"' in s, (f, s)
    for f, s in statements():
        assert not re.search(r"\bs_\w+ m0\b", s), (f, s)
