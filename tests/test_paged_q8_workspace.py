"""Workspaces of prompts over an 8-bit cache (CPU): the room for the bf16 copy is named,
and not insisted on."""

from test_paged_q8_abi import ALIGN, DEVICE, R, WS, fwd, lib, no_gpu, pages  # noqa: F401
from test_abi import _t

MANY = dict(q=_t(b=1, h=8, n=600))   # 2400 rows of a key head for two sequences of 128


def sizes(lib, q, batch, width):  # noqa: F811
    return tuple(f(R(q), R(pages(p=4000)), batch, width)
                 for f in (lib.attn_paged_fwd_q8_workspace_size, lib.attn_paged_fwd_workspace_size))


def test_the_copy_is_named(lib):  # noqa: F811
    copy, rest = sizes(lib, MANY["q"], 2, 40)
    rows = 2 * 40 * 16                                         # of the pages that two tables name
    assert copy - rest == 2 * rows * 2 * 128 * 2 + 512         # and the table of 80 entries, 256 bytes each way
    assert sizes(lib, _t(b=1, h=8, n=500), 2, 40)[0] == sizes(lib, _t(b=1, h=8, n=500), 2, 40)[1]
    # more than 8 D rows a sequence: 256 tokens of four heads are as many
    for d in (64, 128):
        for n, more in ((2 * d, False), (2 * d + 1, True)):
            copy, rest = (f(R(_t(b=1, h=8, n=n, d=d)), R(pages(p=400, d=d)), 1, 40)
                          for f in (lib.attn_paged_fwd_q8_workspace_size, lib.attn_paged_fwd_workspace_size))
            assert (copy > rest) == more
    # sizes without a copy grow with the batch and the width; those with one need not
    for q in (MANY["q"], _t(b=1, h=8, n=40)):
        rest = [[sizes(lib, q, b, w)[1] for w in (4, 40, 400, 4000)] for b in (1, 2, 3, 8, 64)]
        assert all(x == sorted(x) for x in rest) and all(list(x) == sorted(x) for x in zip(*rest))
    assert sizes(lib, MANY["q"], 2, 40)[0] > sizes(lib, MANY["q"], 3, 40)[0]


@no_gpu
def test_a_workspace_without_room_for_the_copy_is_taken(lib):  # noqa: F811
    copy, rest = sizes(lib, MANY["q"], 2, 40)
    kw = dict(MANY, kp=pages(p=4000), width=40, stride=40)
    for n in (copy, copy - 1, rest):
        assert fwd(lib, n=n, **kw) == DEVICE


def test_the_rest_is_insisted_on(lib):  # noqa: F811
    _, rest = sizes(lib, MANY["q"], 2, 40)
    kw = dict(MANY, kp=pages(p=4000), width=40, stride=40)
    assert fwd(lib, n=rest - 1, **kw) == WS
    assert fwd(lib, n=0, **kw) == WS
    assert fwd(lib, ws=None, n=rest, **kw) == WS
    assert fwd(lib, n=rest, ws=0x10010, **kw) == ALIGN
