"""What the kernels' sources have to state, read as text (no GPU needed)."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "gguf_q4_dequant_amd", "csrc", "*")))


def asm_statements(text):
    """(instructions, clobbers) of every asm statement of a C++ source."""
    text = re.sub(r"//[^\n]*", "", text)
    found = []
    for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
        # the statement ends where its parentheses do, strings apart
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if quoted:
                at += c == "\\"
                quoted = c != '"'
            elif c == '"':
                quoted = True
            else:
                depth += (c == "(") - (c == ")")
            at += 1
        body = text[m.end():at - 1]
        parts, string = [""], r'"(?:[^"\\]|\\.)*"'
        for token in re.findall(string + r"|::|[^\"]", body):  # the colons between the parts, not those in strings
            if token in (":", "::"):
                parts += [""] * len(token)
            else:
                parts[-1] += token
        code = " ".join(re.findall(string, parts[0]))
        clobbers = re.findall(r'"(\w+)"', parts[3]) if len(parts) > 3 else []
        found.append((code, clobbers))
    return found


def test_asm_statements_are_taken_apart():
    got = asm_statements('asm volatile("s_mov_b32 m0, %1\\n\\tx %0" ::"v"(a(b)), "s"(c) : "memory", "m0"); asm volatile("" ::: "memory");'
                         'asm volatile("" : "+v"(z));')
    assert got == [('"s_mov_b32 m0, %1\\n\\tx %0"', ["memory", "m0"]), ('""', ["memory"]), ('""', [])]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_assembly_that_writes_m0_names_it(path):
    for code, clobbers in asm_statements(open(path).read()):
        if re.search(r"\bm0\b", code):
            assert "m0" in clobbers, code
