"""Workspace sizes of the paged attention (CPU).  A size is asked for before the
call is checked, so it has to be safe for any numbers: 0 where the call itself
would be refused, which then says why."""

import ctypes
import os
import subprocess
import sys

import pytest

from test_abi import _t
from test_paged_abi import DEVICE, SHAPE, UNSUP, WS, _pages, decode, fwd, lib, no_gpu  # noqa: F401

R = ctypes.byref
ALIGN = -4
BIG = 1 << 62


PRELUDE = """
import ctypes, sys
sys.path[:0] = ["tests", "."]
from test_abi import _t
from test_paged_abi import _pages, decode, fwd
from long_sequence_exact_gb300 import _lib
lib, R = _lib.load(), ctypes.byref
"""


def in_child(body):
    """The lines that `body` prints where a signal ends no more than a child."""
    r = subprocess.run([sys.executable, "-c", PRELUDE + body], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    return r.stdout.split("\n")[:-1]


def test_too_many_rows_behind_a_prefix(lib):  # noqa: F811
    got = in_child("""
for per in (65, 128, 129, 192):
    for b in (1, 2, 500):
        for prefix_len in (0, 100, 100000):
            q, kp = _t(b=b, h=per, n=1), _pages(h=1)
            print(lib.attn_paged_decode_workspace_size(R(q), R(kp), 4000, prefix_len),
                  decode(lib, q=q, kp=kp, width=4000, stride=4000, prefix=0x4000, prefix_len=prefix_len), flush=True)
""")
    assert got == [f"0 {UNSUP}"] * 36


# what the sizes are asked with, and what the call with the same numbers says
DECODE_REFUSED = [
    (dict(q=dict(d=0), kp=dict(d=0)), SHAPE),
    (dict(q=dict(d=96), kp=dict(d=96)), UNSUP),
    (dict(q=dict(d=64)), SHAPE),
    (dict(q=dict(n=0)), SHAPE),
    (dict(q=dict(n=17)), UNSUP),
    (dict(q=dict(h=7)), SHAPE),
    (dict(q=dict(h=0)), SHAPE),
    (dict(q=dict(b=0)), SHAPE),
    (dict(q=dict(b=-1)), SHAPE),
    (dict(q=dict(b=1 << 16)), UNSUP),
    (dict(kp=dict(page=0)), UNSUP),
    (dict(kp=dict(page=8)), UNSUP),
    (dict(kp=dict(page=24)), UNSUP),
    (dict(kp=dict(page=512)), UNSUP),
    (dict(kp=dict(h=0)), SHAPE),
    (dict(kp=dict(p=0)), SHAPE),
    (dict(kp=dict(p=1 << 31)), UNSUP),
    (dict(width=-1), SHAPE),
    (dict(width=1 << 27), UNSUP),
    (dict(width=BIG), UNSUP),
    (dict(prefix_len=-1), SHAPE),
    (dict(prefix_len=-BIG), SHAPE),
    (dict(prefix_len=1 << 31), UNSUP),
    (dict(prefix_len=BIG), UNSUP),
]


def test_decode_sizes_of_refused_calls(lib):  # noqa: F811
    got = in_child(f"""
for case in {[c for c, _ in DECODE_REFUSED]}:
    q, kp = _t(**{{**dict(b=2, h=8, n=1), **case.get("q", {{}})}}), _pages(**case.get("kp", {{}}))
    width, prefix_len = case.get("width", 4000), case.get("prefix_len", 0)
    print(lib.attn_paged_decode_workspace_size(R(q), R(kp), width, prefix_len),
          decode(lib, q=q, kp=kp, width=width, stride=max(0, width), prefix=0x4000, prefix_len=prefix_len), flush=True)
""")
    assert got == [f"0 {code}" for _, code in DECODE_REFUSED]


FWD_REFUSED = [
    (dict(q=dict(d=0), kp=dict(d=0)), SHAPE),
    (dict(q=dict(d=96), kp=dict(d=96)), UNSUP),
    (dict(q=dict(d=64)), SHAPE),
    (dict(q=dict(n=-1)), SHAPE),
    (dict(q=dict(n=1 << 31)), UNSUP),
    (dict(q=dict(h=7)), SHAPE),
    (dict(q=dict(h=258)), UNSUP),       # 129 heads share a key head
    (dict(q=dict(b=2)), SHAPE),
    (dict(kp=dict(page=0)), UNSUP),
    (dict(kp=dict(page=100)), UNSUP),
    (dict(kp=dict(h=0)), SHAPE),
    (dict(width=-1), SHAPE),
    (dict(width=BIG), UNSUP),
    (dict(batch=0), SHAPE),
    (dict(batch=-BIG), SHAPE),
    (dict(batch=4097), UNSUP),
    (dict(batch=BIG), UNSUP),
]


def test_prompt_sizes_of_refused_calls(lib):  # noqa: F811
    got = in_child(f"""
for case in {[c for c, _ in FWD_REFUSED]}:
    q, kp = _t(**{{**dict(b=1, h=8, n=40), **case.get("q", {{}})}}), _pages(**case.get("kp", {{}}))
    width, batch = case.get("width", 4000), case.get("batch", 2)
    print(lib.attn_paged_fwd_workspace_size(R(q), R(kp), batch, width),
          fwd(lib, q=q, kp=kp, width=width, stride=max(0, width), batch=batch), flush=True)
""")
    assert got == [f"0 {code}" for _, code in FWD_REFUSED]


def test_sizes_without_views(lib):  # noqa: F811
    q, kp = _t(b=2, h=8, n=1), _pages()
    for f in (lib.attn_paged_decode_workspace_size, lib.attn_paged_fwd_workspace_size):
        assert f(None, R(kp), 4, 4) == 0
        assert f(R(q), None, 4, 4) == 0


@no_gpu
@pytest.mark.parametrize("b,prefix_len", [(2, 0), (2, 100), (8, 100), (9, 100), (64, 5000)])
def test_decode_workspaces(lib, b, prefix_len):  # noqa: F811
    """Runs, and behind a prefix both layouts (4 rows a sequence and key head: up
    to 32 rows, and more): exactly what is needed, and 256-byte aligned."""
    q, kp, wide = _t(b=b, h=8, n=1), _pages(), dict(width=4000, stride=4000)
    need = lib.attn_paged_decode_workspace_size(R(q), R(kp), 4000, prefix_len)
    assert need > 0
    kw = dict(q=q, kp=kp, prefix=0x4000, prefix_len=prefix_len, **wide)
    assert decode(lib, ws=None, n=need, **kw) == WS
    assert decode(lib, n=need - 1, **kw) == WS
    assert decode(lib, ws=0x10010, n=need, **kw) == ALIGN
    assert decode(lib, n=need, **kw) == DEVICE


@no_gpu
def test_clusters_need_no_workspace(lib):  # noqa: F811
    q, kp = _t(b=2, h=8, n=1), _pages()
    assert lib.attn_paged_decode_workspace_size(R(q), R(kp), 4, 0) == 0
    assert decode(lib, ws=None, n=0) == DEVICE


@no_gpu
@pytest.mark.parametrize("width", [4, 4000])
def test_prompt_workspaces(lib, width):  # noqa: F811
    q, kp = _t(b=1, h=8, n=40), _pages()
    need = lib.attn_paged_fwd_workspace_size(R(q), R(kp), 2, width)
    assert need > 0
    kw = dict(q=q, kp=kp, width=width, stride=width)
    assert fwd(lib, ws=None, n=need, **kw) == WS
    assert fwd(lib, n=need - 1, **kw) == WS
    assert fwd(lib, ws=0x10010, n=need, **kw) == ALIGN
    assert fwd(lib, n=need, **kw) == DEVICE


def test_python_sizes_of_refused_calls(lib):  # noqa: F811
    """The Python face asks for the size first, whether or not a workspace is
    given; the refusal is the call's (made before a device is touched)."""
    got = in_child("""
import torch
from long_sequence_exact_gb300 import paged
paged._device, paged._stream = (lambda *t: 0), (lambda dev: 0)
z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
i = lambda *s: torch.zeros(s, dtype=torch.int32)
kp = z(8, 1, 16, 128)
for per, nq in ((65, 1), (128, 1), (129, 1), (192, 1), (64, 3)):
    q = z(2, per, nq, 128)
    print(paged.paged_decode_workspace_size(q, kp, 4000, 100))
    for ws in (None, torch.zeros(512, dtype=torch.uint8)):
        try:
            paged.paged_decode(q, kp, kp, i(2, 4000), i(2), prefix_table=i(7), prefix_len=100, workspace=ws)
        except _lib.LsxError as e:
            print(e.code, flush=True)
q = z(1, 129, 9, 128)
print(paged.paged_fwd_workspace_size(q, kp, 2, 4000))
try:
    paged.paged_fwd(q, kp, kp, i(2, 4000), i(2), i(3))
except _lib.LsxError as e:
    print(e.code)
""")
    assert got == ["0", str(UNSUP), str(UNSUP)] * 5 + ["0", str(UNSUP)]
