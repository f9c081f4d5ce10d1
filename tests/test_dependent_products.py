"""The 4-bit products' kernel that is launched as a programmatic dependent of the one that scales x, read as text (no GPU): what the
kernel before it writes is read behind the wait only, by loads that may not be moved or cached as read-only."""
import re

import pytest

from test_dependent_launches import body, sources


def dependents(text):
    """Names of the kernels that a launch with programmatic serialization takes, other than through launch_after."""
    found = set()
    for at in re.finditer(r"cudaLaunchAttributeProgrammaticStreamSerialization", text):
        start = text.rfind("\n}\n", 0, at.start())
        found |= set(re.findall(r"\b(q4_\w+_kernel)\s*<", text[start:at.start()]))
    return sorted(found)


def test_the_kernel_is_found():
    assert dependents(sources()) == ["q4_tc_kernel"]


def test_no_thread_ends_before_the_last_barrier():
    """Some threads of every CTA wait for the kernel before, and all meet at a barrier behind that: none ends without it."""
    code = body(sources(), "q4_tc_kernel")
    assert not re.search(r"\breturn;|\bexit\b", re.sub(r"\[&\][^;]*?\{.*?\n        \};", "", code, flags=re.S))
    wait = [m.start() for m in re.finditer(r"grid_dependency_wait\(\)", code)]
    assert len(wait) == 2 and code.rindex("__syncthreads()") > wait[-1]


@pytest.mark.parametrize("name", ["x_exponents", "x_map"])
def test_what_the_kernel_before_writes(name):
    text = sources()
    code = body(text, "q4_tc_kernel")
    head = re.search(r"q4_tc_kernel\(([^{]*?)\)\s*\{", text[text.index("__global__ void __launch_bounds__(Tc<"):], re.S).group(1)
    assert not re.search(r"__restrict__\s+%s\b" % name, head)
    if name == "x_exponents":                        # read once, behind the wait, as volatile
        uses = [m.start() for m in re.finditer(r"\bx_exponents\b", code)]
        assert len(uses) == 1 and code.rindex("grid_dependency_wait()", 0, uses[0]) > 0 and "volatile" in code[uses[0] - 60:uses[0]]
    else:                                            # asked for in load_x alone, whose first calls stand behind the first wait
        calls = [m.start() for m in re.finditer(r"\bload_x\(", code)]
        assert code.index("grid_dependency_wait()") < calls[0]
