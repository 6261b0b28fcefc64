"""How calls of the attention step are cut, on the host (nothing here touches a GPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_call_reads_the_environment():
    """A call is cut by its arguments alone: a variable of the process neither changes its bits nor ends it."""
    csrc = os.path.join(ROOT, "lora_serving_amd", "csrc", "**")
    files = [p for kind in ("*.cpp", "*.h", "*.hip") for p in glob.glob(os.path.join(csrc, kind), recursive=True)]
    assert len(files) > 10
    for path in sorted(files):
        with open(path) as f:
            assert not re.search(r"\b(secure_)?getenv\b|\benviron\b", f.read()), path


def test_numbers_of_groups_that_do_not_fit_are_refused():
    """64 lanes count the groups in equal runs, in 32 bits: 2^31 - 1 of them plus a run's remainder would not fit."""
    from lora_serving_amd import mlora as m
    from tests.test_attention_prefix_host import call, size
    sizes = lambda n: size(m, 100, 20, n, 32, 8, 128, 5, 4000, 2000)  # noqa: E731
    for n in (1 << 30, (1 << 31) - 64, (1 << 31) - 1):
        assert call(m, groups=n) == m.MLORA_ERR_UNSUPPORTED
        assert sizes(n) == 0
    assert call(m, groups=(1 << 30) - 1) == m.MLORA_ERR_WORKSPACE
    assert sizes((1 << 30) - 1) > 0
