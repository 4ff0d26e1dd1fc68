"""A kernel that may start before the launch ahead of it has ended reports no error
before it has waited for that launch, which clears the status word: the report
could be cleared with it.  Read from the sources: no call can show it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deterministic_attn_backward_gb300",
                    "csrc")


def kernels(name):
    """(name, body) of the file's kernels."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for part in re.split(r"__global__", text)[1:]:
        head = re.sub(r"__launch_bounds__\([^()]*(\([^()]*\))?[^()]*\)", "", part)
        yield re.search(r"void\s+(\w+)\s*\(", head).group(1), part[:part.find("\n}\n")]


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith(".cu")))
def test_no_report_before_the_wait(name):
    for kernel, body in kernels(name):
        if "grid_wait()" in body and "raise_error(" in body:
            assert body.index("grid_wait()") < body.index("raise_error("), kernel
