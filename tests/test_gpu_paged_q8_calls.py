"""How calls over an 8-bit cache run: which kernels, in which workspaces."""

import ctypes

import pytest
import torch

import long_sequence_exact_gb300 as lsx
from long_sequence_exact_gb300 import _lib
from test_gpu_paged import done, ints
from test_gpu_paged_q8_attention import prompt_case

pytestmark = pytest.mark.gpu
DEV = "cuda"
MANY = (8, 2, 64, 32, [(700, 300), (0, 200)])   # 8 D rows a sequence and key head and more: by a copy


def kernels(fn):
    """The kernels that the library's timing counts in a call: {name: launches}."""
    lib, buf = _lib.load(), ctypes.create_string_buffer(4096)
    lib.lsx_timing_reset()
    lib.lsx_timing_enable(1)
    try:
        fn()
        torch.cuda.synchronize()
        lib.lsx_timing_report(buf, 4096)
    finally:
        lib.lsx_timing_enable(0)
        lib.lsx_timing_reset()
    return {x.split()[0]: int(x.split()[1]) for x in buf.value.decode().strip().splitlines()}


def test_the_copy_is_timed_as_itself():
    q, c, table, lens, cu = prompt_case(*MANY)
    got = kernels(lambda: lsx.paged_fwd_q8(q, *c.parts, table, ints(lens), ints(cu)))
    assert got["page_widen"] == 1 and "page_read" not in got
    n = int(lens[0])
    got = kernels(lambda: lsx.page_read_q8(*c.parts, table[:1], ints([0]), ints([0, n]), n))
    assert got == {"page_read": 1}
    assert done() == 0
