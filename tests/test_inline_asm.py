"""CPU test of the kernels' inline assembly: a fixed register that a statement writes is named as overwritten."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_gated_delta_08_amd", "csrc")


def statements(text):
    """The text of each asm statement, from its opening bracket to the closing one."""
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            depth += 0 if quoted else (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


def test_written_registers_are_named():
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*")):
        for s in statements(open(path, encoding="utf-8").read()):
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', s.split(":")[0])).replace("\\n", "\n").replace("\\t", " ")
            clobbers = re.findall(r'"(\w+)"', s.rsplit(":", 1)[1]) if s.count(":") >= 3 else []
            for line in code.splitlines():
                words = line.split()
                if len(words) > 1 and re.fullmatch(r"m0|vcc|exec|scc", words[1].rstrip(",")):
                    seen += 1
                    assert words[1].rstrip(",") in clobbers, (path, s)
    assert seen   # the loads into LDS set m0
