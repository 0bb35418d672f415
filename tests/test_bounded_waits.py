"""Roles that leave their loops when a wait runs out meet in no barrier before the
block's end: one that has left would not come to it (CPU: read from the sources)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_sequence_exact_gb300", "csrc")


def kernel(name, file):
    """The text of a kernel, from its name to the next line that ends a function."""
    text = open(os.path.join(CSRC, file)).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = text.index(name + "(const __grid_constant__")
    return text[at:text.index("\n}\n", at)]


def test_prompt_kernel_has_barriers_at_its_ends_alone():
    body = kernel("paged_fwd_kernel", "paged_fwd.cu")
    assert "mbar_wait" in body and "bar.sync" not in body and "barrier.sync" not in body
    parts = body.split("__syncthreads()")
    assert len(parts) == 3
    assert "mbar_wait" not in parts[0] and "mbar_wait" not in parts[2]  # all waits are between the two


@pytest.mark.parametrize("file,name", [("paged_decode.cu", "paged_decode_kernel"),
                                       ("paged_decode_q8.cu", "paged_decode_q8_kernel")])
def test_decode_kernels_do_not_leave_by_a_wait_before_a_barrier(file, name):
    """Their compute warps meet at each unit's end, so a wait that ran out must not end
    their loop: its result is not looked at."""
    body = kernel(name, file)
    loop = body[body.index("computes && it < n_steps"):] if "computes && it" in body else body
    waits = re.findall(r"[^;{}]*mbar_wait\(&sh\.full\[[^;]*;", loop)
    assert waits and all(w.strip().startswith("mbar_wait") for w in waits)
