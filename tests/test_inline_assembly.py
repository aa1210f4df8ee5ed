"""Inline assembly says which registers it changes: the compiler would not see it otherwise."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def statements():
    for path in sorted(glob.glob(os.path.join(ROOT, "block_quantized_communication_amd", "csrc", "*.h*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", text, re.S):
            parts = re.split(r"(?<!:):(?!:)", m.group(1).replace("::", ": :"))
            yield os.path.basename(path), parts[0], parts[3] if len(parts) > 3 else ""


def test_fixed_registers_are_named():
    """m0, vcc and exec where an instruction writes them, that is, names them first."""
    found = 0
    for path, code, clobbers in statements():
        for register in ("m0", "vcc", "exec"):
            if re.search(r"(?:^|\\t|\")\s*[sv]_\w+\s+" + register + r"\b", code):
                found += 1
                assert f'"{register}"' in clobbers, (path, code)
    assert found >= 2
