"""Loads through the read-only path (`__ldg`) are for data that nothing writes while
the kernel runs.  A kernel that may start before the launch ahead of it has ended
(it calls grid_wait()) may load only the caller's inputs that way, not what that
launch makes.  Read from the sources: outputs cannot show it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deterministic_attn_backward_gb300",
                    "csrc")
INPUTS = {"p.limit"}          # written by no launch of the library


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))))
def test_only_inputs_are_loaded_as_read_only(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    if "grid_wait()" not in text:
        return
    loaded = {m.group(1) for m in re.finditer(r"__ldg\(\s*([\w.\->]+)", text)}
    assert loaded <= INPUTS
