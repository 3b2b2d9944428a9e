"""What the kernels' inline assembly has to tell the compiler."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_get_dispatch_03_amd", "csrc")


def asm_statements(text):
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            if not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text[m.end():at - 1]


def test_a_written_m0_is_a_clobber():
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*.h*")):
        for asm in asm_statements(open(path).read()):
            if re.search(r"\bm0,", asm):
                seen += 1
                assert re.search(r':\s*(?:"\w+"\s*,\s*)*"m0"', asm.split("lds\"", 1)[-1]), (os.path.basename(path), asm)
    assert seen == 3
