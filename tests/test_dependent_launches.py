"""Kernels that are launched as programmatic dependents of the one before them, read as text (no GPU): none of their threads may
end before it has waited for that kernel's end.  The wait is what orders them; a grid whose threads have all ended without it
counts as finished although the kernel before it still runs."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_03_gb300", "csrc")


def sources():
    text = "\n".join(open(f).read() for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))))
    return re.sub(r"//[^\n]*", "", text)


def dependents(text):
    """Names of the kernels handed to launch_after."""
    return sorted(set(re.findall(r"launch_after\((?:[^;]*?)\b(attend_\w+_kernel)\s*<", text, re.S)))


def body(text, kernel):
    at = re.search(r"__global__[^;{]*?\b%s\(" % kernel, text).end()
    start = text.index("{", text.index(")", at))
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(kernel)


def test_the_kernels_are_found():
    assert dependents(sources()) == ["attend_join_kernel", "attend_merge_kernel", "attend_tc_kernel"]


@pytest.mark.parametrize("kernel", ["attend_join_kernel", "attend_merge_kernel", "attend_tc_kernel"])
def test_no_thread_ends_before_the_wait(kernel):
    code = body(sources(), kernel)
    assert "grid_dependency_wait()" in code
    before = code[:code.index("grid_dependency_wait()")]
    assert not re.search(r"\breturn\b|\bexit\b", before)
