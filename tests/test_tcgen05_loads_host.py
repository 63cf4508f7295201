"""tcgen05.ld is asynchronous: its registers hold nothing before tcgen05.wait::ld. The compiler
may copy or spill registers between two asm statements, so a load whose wait is another
statement can leave values (or take registers, addresses among them, that the load still writes).
Every load in the sources therefore shares its statement with a wait behind it."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "random_feature_linear_b200", "csrc")


def asm_statements(text):
    """The argument texts of all asm statements."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b\s*(?:volatile\s*)?\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if quoted and c == "\\":
                i += 1
            elif c == '"':
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


def test_loads_and_their_wait_are_one_statement():
    loads = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for s in asm_statements(open(path).read()):
            if "tcgen05.ld" in s:
                loads += 1
                assert s.rfind("tcgen05.wait::ld") > s.rfind("tcgen05.ld"), (path, s[:80])
    assert loads > 0
