"""How calls of the attention step are cut, on the host (nothing here touches a GPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_call_reads_the_environment():
    """A call is cut by its arguments alone: a variable of the process neither changes its bits nor ends it."""
    files = [p for kind in ("*.cpp", "*.h", "*.hip") for p in glob.glob(os.path.join(ROOT, "lora_serving_amd", "csrc", "**", kind),
                                                                         recursive=True)]
    assert len(files) > 10
    for path in sorted(files):
        with open(path) as f:
            assert not re.search(r"\b(secure_)?getenv\b|\benviron\b", f.read()), path
