"""The 8-bit training operators on the CPU: what their sources, header and argument checks promise."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_mixed_precision_rank_amd", "csrc")


def inline_asm():
    """(file, text) of every asm statement of the library's device sources, up to its closing bracket."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".hip", ".h")):
            continue
        src = open(os.path.join(CSRC, name), encoding="utf-8").read()
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", src):
            depth, i = 1, m.end()
            quoted = False
            while depth:
                c = src[i]
                if c == '"' and src[i - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                i += 1
            yield name, src[m.end():i - 1]


def test_loads_to_lds_take_m0_as_an_operand():
    """A statement that writes m0 by itself, without the compiler's knowledge, could land between the compiler's own
    write and its use; and a load to LDS has to have m0 from somewhere."""
    found = 0
    for name, text in inline_asm():
        template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split(" : ")[0]))
        for instruction in template.replace("\\t", "").split("\\n"):
            assert not re.match(r"\s*\w+\s+m0\b", instruction), (name, instruction)
            if re.search(r"\blds$", instruction):
                assert '"{m0}"' in text, (name, instruction)
                found += 1
    assert found == 2
