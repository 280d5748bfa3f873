"""Copies from memory into LDS take their LDS address from M0, and gfx950 needs one
instruction between a scalar write of M0 and the copy that reads it. Inline asm gets
no such wait from the compiler: every block has to hold it itself (read from the
sources, no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_mixture_experts_05_amd", "csrc")


def asm_blocks():
    """(file, instructions) of every inline asm statement of the sources."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            body = re.match(r'(?:\s*"(?:[^"\\]|\\.)*")+', text[m.end():]).group(0)
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body))
            yield os.path.basename(path), [i.strip() for i in re.split(r"\\n|\\t|;", code) if i.strip()]


def test_copies_wait_for_m0():
    copies = 0
    for name, code in asm_blocks():
        for i, ins in enumerate(code):
            if not re.match(r"(global|buffer)_load_lds", ins):
                continue
            copies += 1
            sets = [j for j in range(i) if re.match(r"s_\w+\s+m0\b", code[j])]
            assert sets, f"{name}: {ins} relies on an M0 set outside its block"
            assert i - sets[-1] >= 2, f"{name}: nothing between the write of M0 and {ins}"
    assert copies >= 3
