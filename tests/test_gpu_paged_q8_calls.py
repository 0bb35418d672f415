"""How calls over an 8-bit cache run: which kernels, in which workspaces."""

import ctypes

import pytest
import torch

import long_sequence_exact_gb300 as lsx
import paged_ref as P
from long_sequence_exact_gb300 import _lib
from test_gpu_paged import check_prompt, done, ints
from test_gpu_paged_q8_attention import prompt_case

pytestmark = pytest.mark.gpu
DEV = "cuda"
MANY = (8, 2, 64, 32, [(700, 300), (0, 200)])   # more than 8 D rows a sequence and key head: by a copy


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


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_of_many_rows_without_room_for_a_copy(d, out_dtype):
    """The workspace decides: with room for the copy it is made, with a byte less, or with
    the size without it, the tiles are widened where they are used, bit for bit alike; NaN
    behind the workspace's end is not read, and stays."""
    q, c, table, lens, cu = prompt_case(8, 2, d, 32, [(700, 300), (0, 300)], tail=3)
    dense = c.dense()
    o_ref, l_ref = P.fwd(q, *dense, table, lens, cu)
    full, rest = (lsx.paged_fwd_q8_workspace_size(q, c.kp, 2, table.shape[1], copy=x) for x in (True, False))
    assert full > rest > 0
    outs = []
    for n in (full, full - 1, rest):
        ws = torch.full((full + 512,), 255, dtype=torch.uint8, device=DEV)
        ws = ws[(-ws.data_ptr()) % 256:]
        o, lse = torch.full(q.shape, 7.0, dtype=out_dtype, device=DEV), torch.full(q.shape[:3], 7.0, device=DEV)
        got = kernels(lambda: lsx.paged_fwd_q8(q, *c.parts, table, ints(lens), ints(cu), out=o, lse=lse, workspace=ws[:n]))
        assert ("page_widen" in got) == (n == full) and done() == 0
        assert bool((ws[n:] == 255).all())
        bits = ((2.0 ** -8, 2.0 ** -16) if n == full else (2.0 ** -11, 2.0 ** -22))[out_dtype is torch.float32]
        tol, tol_lse = P.tolerances(q, *dense, bits, out_dtype)
        check_prompt(o, lse, o_ref, l_ref, tol, tol_lse)
        outs.append((o, lse))
    assert all(torch.equal(a, b) for a, b in zip(outs[1], outs[2]))


@pytest.mark.parametrize("width", [0, 400])
@pytest.mark.parametrize("tokens", [256, 257])
def test_the_border_of_the_copy(tokens, width):
    """As many rows as 8 D a sequence are worked on in place, which is faster there and
    keeps P to f16; one token more by a copy, whose pages are numbered by sequence and
    column or, behind a wide table, as in the pool."""
    q, c, table, lens, cu = prompt_case(32, 8, 128, 64, [(3000, tokens)])
    if width:
        table = torch.cat([table, torch.full((1, width), -1, dtype=torch.int32, device=DEV)], 1)
        assert table.shape[1] > c.kp.shape[0]
    dense = c.dense()
    o_ref, l_ref = P.fwd(q, *dense, table, lens, cu)
    out = []
    got = kernels(lambda: out.extend(lsx.paged_fwd_q8(q, *c.parts, table, ints(lens), ints(cu))))
    assert ("page_widen" in got) == (tokens > 256) and done() == 0
    tol, tol_lse = P.tolerances(q, *dense, 2.0 ** -8 if tokens > 256 else 2.0 ** -11, torch.bfloat16)
    check_prompt(*out, o_ref, l_ref, tol, tol_lse)
