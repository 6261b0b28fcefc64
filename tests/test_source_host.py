"""What the compiler cannot check in the kernels' inline assembly."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def statements():
    for path in sorted(glob.glob(os.path.join(ROOT, "lora_serving_amd", "csrc", "*.h")) +
                       glob.glob(os.path.join(ROOT, "lora_serving_amd", "csrc", "*.hip"))):
        with open(path) as f:
            for asm in re.findall(r"\basm\s+volatile\s*\(.*?\)\s*;", f.read(), re.S):
                yield os.path.basename(path), asm


def test_assembly_names_what_it_overwrites():
    """m0 and scc, which no operand stands for, are among the clobbers of a statement that writes them."""
    writers = 0
    for name, asm in statements():
        code = asm.split("::")[0]
        clobbers = asm.rsplit(":", 1)[-1]
        if re.search(r"\bs_\w+ m0\b", code):
            writers += 1
            assert '"m0"' in clobbers, f"{name}: {asm}"
        if re.search(r"\bs_(add|sub|and|or|xor|lshl|lshr|ashr|cmp)\w*\b", code):
            assert '"scc"' in clobbers, f"{name}: {asm}"
    assert writers        # (the copies straight into LDS)
