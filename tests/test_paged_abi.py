"""Argument checks of the paged entry points (CPU): every refusal is made
before a device is touched.  On a machine without a GPU a call whose arguments
are in order ends with LSX_ERR_DEVICE (-9), having launched nothing."""

import ctypes

import pytest
import torch

from test_abi import _lse, _t

R = ctypes.byref
NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS, DEVICE = -1, -2, -3, -4, -5, -6, -9
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would launch on made-up pointers")


@pytest.fixture(scope="module")
def lib():
    from long_sequence_exact_gb300 import build, _lib
    build.build()
    return _lib.load()


def _pages(p=8, h=2, page=16, d=128, dtype=0, ptr=0x30000):
    return _t(p, h, page, d, dtype, ptr)


def decode(lib, q=None, kp=None, vp=None, table=0x1000, stride=4, width=4, lens=0x2000, prefix=None,
           prefix_len=0, o=None, lse=None, ws=0x10000, n=1 << 40):
    q = q or _t(b=2, h=8, n=1)
    kp = kp or _pages()
    vp = vp or kp
    o = o or _t(b=q.B, h=q.H, n=q.N, d=q.D)
    lse = lse or _lse(q.B, q.H, q.N)
    return lib.attn_paged_decode(R(q), R(kp), R(vp), table, stride, width, lens, prefix, prefix_len,
                                 -1.0, R(o), R(lse), ws, n, None)


def fwd(lib, q=None, kp=None, table=0x1000, stride=4, width=4, lens=0x2000, cu=0x3000, batch=2, o=None,
        lse=None, ws=0x10000, n=1 << 40):
    q = q or _t(b=1, h=8, n=40)
    kp = kp or _pages()
    o = o or _t(b=q.B, h=q.H, n=q.N, d=q.D)
    lse = lse or _lse(q.B, q.H, q.N)
    return lib.attn_paged_fwd(R(q), R(kp), R(kp), table, stride, width, lens, cu, batch, -1.0, R(o),
                              R(lse), ws, n, None)


@no_gpu
def test_calls_in_order_reach_the_device(lib):
    assert decode(lib) == DEVICE
    assert decode(lib, q=_t(b=2, h=8, n=4, d=64), kp=_pages(d=64, page=256)) == DEVICE
    assert decode(lib, prefix=0x4000, prefix_len=100) == DEVICE
    assert decode(lib, o=_t(b=2, h=8, n=1, dtype=1)) == DEVICE      # f32 output
    assert decode(lib, table=None, stride=0, width=0) == DEVICE     # no table: no keys of their own
    assert fwd(lib) == DEVICE
    assert map_(lib) == DEVICE
    assert append(lib) == DEVICE
    assert append(lib, k=_t(b=1, h=2, n=5, dtype=1)) == DEVICE      # f32 rows


@pytest.mark.parametrize("call", [decode, fwd])
def test_attention_refusals(lib, call):
    n = 1 if call is decode else 40
    b = 2 if call is decode else 1
    q = lambda **kw: _t(**{**dict(b=b, h=8, n=n), **kw})  # noqa: E731
    assert call(lib, q=q(dtype=1)) == DTYPE
    assert call(lib, kp=_pages(dtype=1)) == DTYPE
    assert call(lib, q=q(d=64)) == SHAPE                       # head size differs from the cache's
    assert call(lib, q=q(h=7)) == SHAPE                        # heads not a multiple
    assert call(lib, q=q(ptr=0x10008)) == ALIGN
    assert call(lib, q=q(strides=(8 * 132, 130, 130))) == ALIGN
    assert call(lib, o=_t(b=b, h=8, n=n, d=64)) == SHAPE
    assert call(lib, o=_t(b=b, h=8, n=n, ptr=0x10004)) == ALIGN
    assert call(lib, lse=_lse(b, 8, n + 1)) == SHAPE
    bad = _lse(b, 8, n)
    bad.dtype = 0
    assert call(lib, lse=bad) == DTYPE
    for page in (8, 24, 100, 512):
        assert call(lib, kp=_pages(page=page)) == UNSUP
    assert call(lib, q=q(d=96), kp=_pages(d=96)) == UNSUP
    assert call(lib, kp=_pages(p=1 << 31)) == UNSUP
    assert call(lib, kp=_pages(ptr=0)) == NULL
    assert call(lib, table=None) == NULL
    assert call(lib, lens=None) == NULL
    assert call(lib, lens=0x2002) == ALIGN
    assert call(lib, table=0x1001) == ALIGN
    assert call(lib, stride=3) == SHAPE                        # rows of the table would overlap
    assert call(lib, width=-1) == SHAPE
    assert call(lib, stride=1 << 27, width=1 << 27) == UNSUP   # 2^31 keys a sequence


def test_attention_workspaces(lib):
    # what is needed is asked for; less, none or a misaligned one is refused
    q, kp = _t(b=2, h=8, n=1), _pages()
    need = lib.attn_paged_decode_workspace_size(R(q), R(kp), 4, 0)
    if need:
        assert decode(lib, ws=None, n=need) == WS
        assert decode(lib, n=need - 1) == WS
        assert decode(lib, ws=0x10010) == ALIGN
    q = _t(b=1, h=8, n=40)
    need = lib.attn_paged_fwd_workspace_size(R(q), R(kp), 2, 4)
    if need:
        assert fwd(lib, ws=None, n=need) == WS
        assert fwd(lib, n=need - 1) == WS
        assert fwd(lib, ws=0x10010) == ALIGN


def test_decode_refusals(lib):
    assert decode(lib, vp=_pages(p=7)) == SHAPE
    assert decode(lib, q=_t(b=2, h=8, n=17)) == UNSUP          # 4 heads x 17 tokens > 64 rows
    assert decode(lib, q=_t(b=2, h=8, n=0)) == SHAPE
    assert decode(lib, prefix_len=-1) == SHAPE
    assert decode(lib, prefix=None, prefix_len=1) == NULL
    assert decode(lib, prefix=0x4002, prefix_len=1) == ALIGN
    assert decode(lib, prefix=0x4000, prefix_len=1 << 31) == UNSUP


def test_fwd_refusals(lib):
    assert fwd(lib, cu=None) == NULL
    assert fwd(lib, cu=0x3001) == ALIGN
    assert fwd(lib, batch=0) == SHAPE
    assert fwd(lib, batch=4097) == UNSUP
    assert fwd(lib, q=_t(b=2, h=8, n=40)) == SHAPE             # packed tokens have no batch
    assert fwd(lib, q=_t(b=1, h=258, n=40), kp=_pages(h=2)) == UNSUP  # 129 heads share a key head
    assert fwd(lib, q=_t(b=1, h=8, n=0)) == 0                  # nothing to do


def map_(lib, ctx=0x1000, new=0x1100, batch=3, free=0x1200, n_free=9, page=16, table=0x2000, stride=5,
         width=5, slots=0x3000, n=7, cu=0x4000, lens=0x4100, taken=0x4200):
    return lib.attn_page_map(ctx, new, batch, free, n_free, page, table, stride, width, slots, n, cu,
                             lens, taken, None)


def test_map_refusals(lib):
    for name in ("ctx", "new", "free", "table", "slots", "cu", "lens", "taken"):
        assert map_(lib, **{name: None}) == NULL, name
        assert map_(lib, **{name: 0x1002}) == ALIGN, name
    assert map_(lib, slots=0x3004) == ALIGN                    # 64-bit slots
    assert map_(lib, batch=0) == SHAPE
    assert map_(lib, batch=4097) == UNSUP
    assert map_(lib, n_free=-1) == SHAPE
    assert map_(lib, n=-1) == SHAPE
    assert map_(lib, stride=4) == SHAPE
    for page in (0, 8, 48, 512):
        assert map_(lib, page=page) == UNSUP
    # outputs over inputs: blocks that still read them would see what others wrote
    assert map_(lib, lens=0x1000) == UNSUP                     # lengths updated in place
    assert map_(lib, cu=0x1104) == UNSUP
    assert map_(lib, taken=0x1220) == UNSUP                    # the last free page
    assert map_(lib, slots=0x11e0) == UNSUP                    # runs into the free pages
    assert map_(lib, table=0xfc8) == UNSUP                     # 15 entries: one in the lengths


def append(lib, k=None, v=None, slots=0x5000, kp=None, vp=None):
    k = k or _t(b=1, h=2, n=5)
    return lib.attn_page_append(R(k), R(v or k), slots, R(kp or _pages()), R(vp or _pages()), None)


def test_append_refusals(lib):
    assert append(lib, v=_t(b=1, h=2, n=5, dtype=1)) == DTYPE
    assert append(lib, v=_t(b=1, h=2, n=6)) == SHAPE
    assert append(lib, k=_t(b=2, h=2, n=5)) == SHAPE
    assert append(lib, k=_t(b=1, h=4, n=5)) == SHAPE
    assert append(lib, k=_t(b=1, h=2, n=5, d=64)) == SHAPE
    assert append(lib, kp=_pages(dtype=1)) == DTYPE
    assert append(lib, vp=_pages(page=32)) == SHAPE
    assert append(lib, slots=None) == NULL
    assert append(lib, slots=0x5004) == ALIGN
    assert append(lib, k=_t(b=1, h=2, n=5, ptr=0x10008)) == ALIGN
    assert append(lib, k=_t(b=1, h=2, n=0)) == 0


def test_page_status_is_named(lib):
    from long_sequence_exact_gb300 import _lib
    assert _lib.STATUS[-10] == "LSX_ERR_PAGE"
    assert "page" in lib.lsx_status_string(-10).decode()


def test_python_argument_checks():
    from long_sequence_exact_gb300 import paged
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    assert paged._table(i(3, 5), 3)[1:] == (5, 5)
    assert paged._table(i(3, 8)[:, :5], 3)[1:] == (8, 5)
    with pytest.raises(TypeError):
        paged._table(i(3, 5).long(), 3)
    with pytest.raises(ValueError):
        paged._table(i(4, 5), 3)
    with pytest.raises(ValueError):
        paged._table(i(5, 3).t(), 3)
    with pytest.raises(TypeError):
        paged._ints(i(3).float(), "kv_lens")
    with pytest.raises(ValueError):
        paged._ints(i(3), "kv_lens", 4)
    with pytest.raises(ValueError):
        paged._ints(i(6)[::2], "kv_lens")
