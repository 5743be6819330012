"""What the kernels' sources have to keep and no run can show without a race."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_gemv_packed_b200", "csrc")


def dependent_kernels():
    """(file, kernel, body) of the kernels in files that launch theirs with launch_dependent."""
    found = []
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read() if f.endswith(".cu") else ""
        if "launch_dependent(" not in text:
            continue
        for part in re.split(r"\b__global__\b", text)[1:]:
            head, body = part[:part.index("\n}\n")].split("{\n", 1)
            found.append((f, re.findall(r"(\w+)\(", head)[-1], re.sub(r"//[^\n]*", "", body)))
    return found


def test_every_dependent_kernel_is_found():
    assert {k for _, k, _ in dependent_kernels()} == {"attn_kernel", "attn_join_kernel", "kv_write_kernel", "kv_read_kernel",
                                                      "rmsnorm_kernel"}


@pytest.mark.parametrize("file,kernel,body", dependent_kernels(), ids=lambda x: x if len(x) < 40 else "")
def test_dependents_are_released_after_the_wait(file, kernel, body):
    """A kernel that releases its dependents before it has waited lets an overlapping GEMV read its weights while
    kernels several launches back still write them."""
    assert body.count("grid_dependency_wait()") == 1 and body.count("grid_launch_dependents()") == 1
    assert body.index("grid_dependency_wait()") < body.index("grid_launch_dependents()"), (file, kernel)
    before = body[:body.index("grid_dependency_wait()")]
    assert not re.search(r"\bif\b|\breturn\b|\bfor\b|\bwhile\b", before), "every thread waits"
