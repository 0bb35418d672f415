"""Caches kept in pages: page maps, cache writes and the attention that reads them.

The pool is two bf16 views k_pages, v_pages [P, Hkv, page, D] (any strides, D
contiguous; page a power of two from 16 to 256).  Storage laid out
[P, page, Hkv, D] is passed as ``pages.transpose(1, 2)``.  Position i of
sequence b is row i % page of page block_table[b, i // page].  Lengths, tables
and slots are CUDA tensors that the kernels read when they run, so a step can
be captured in a CUDA graph and replayed with new contents.

One serving step:

    slots, cu, kv_lens, taken = page_map(block_table, ctx_lens, new_lens,
                                         free_pages, page, n_tokens)
    page_append(k, v, k_pages, v_pages, slots)             # every layer
    o, lse = paged_fwd(q, k_pages, v_pages, block_table, kv_lens, cu)
    # or, with one new token per sequence:
    o, lse = paged_decode(q, k_pages, v_pages, block_table, kv_lens)

Caches of 8 bits (half the bytes) have calls of their own, page_append_q8,
page_read_q8, paged_decode_q8 and paged_fwd_q8: pages float8_e4m3fn and, of every row,
one power of two in k_scales, v_scales uint8 [P, Hkv, page] (2^(byte - 127); a row's
bytes next to each other, 16-byte aligned).  Tables, slots and lengths are the same:

    page_append_q8(k, v, k_pages, k_scales, v_pages, v_scales, slots)
    o, lse = paged_decode_q8(q, k_pages, k_scales, v_pages, v_scales, block_table, kv_lens)
    k, v = page_read_q8(k_pages, k_scales, v_pages, v_scales, block_table, first, cu, n)

Tensors live on the current CUDA device; calls are enqueued on the current
stream.  A workspace, where one is given, belongs to one call (or one replay of a
graph) at a time.  Inference only: no gradients are recorded.  A page number, slot or
length outside the cache is skipped on the device and reported by
``sync_status`` (LSX_ERR_PAGE).
"""

from __future__ import annotations

import ctypes
import struct
import threading

import torch

from . import _lib
from ._lib import LSX_BF16, LSX_E4M3, LSX_E8M0, LSX_F32, LsxTensor, check, load

_I32, _I64, _F32, _BF16, _U8 = (torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.uint8)

# One decode step is a call per layer: the views of a call are packed with one
# struct.pack_into into a buffer of the calling thread, which the library reads
# before it returns (a ctypes structure per view costs the call several
# microseconds more).
_VIEW = struct.calcsize("Pii7q")
assert _VIEW == ctypes.sizeof(LsxTensor)
_PACK = {n: struct.Struct("Pii7q" * n) for n in (2, 4, 5, 6, 7)}
_KINDS = {_BF16: LSX_BF16, _F32: LSX_F32}
_KINDS8 = {**_KINDS, torch.float8_e4m3fn: LSX_E4M3, _U8: LSX_E8M0}


class _Views(threading.local):
    def __init__(self):
        self.buf = ctypes.create_string_buffer(_VIEW * max(_PACK))
        self.at = ctypes.addressof(self.buf)


_views = _Views()


def _pack(*tensors, kinds=_KINDS):
    """Addresses of the lsx_tensor views of [B, H, N, D] tensors (D contiguous)
    or [B, H, N] ones (an LSE, the exponents of 8-bit rows), valid until the thread's next _pack."""
    fields = []
    for t in tensors:
        kind = kinds.get(t.dtype)
        if kind is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
        shape, stride = t.shape, t.stride()
        if len(shape) == 4:
            b, h, n, d = shape
            sb, sh, sn, sd = stride
            if sd != 1 and d > 1:
                raise ValueError("the last dimension must be contiguous")
        elif len(shape) == 3:
            b, h, n = shape
            sb, sh, sn = stride
            d = 1
        else:
            raise ValueError("expected a [B, H, N, D] or [B, H, N] tensor")
        fields += (t.data_ptr(), kind, 0, b, h, n, d, sb, sh, sn)
    views = _views
    _PACK[len(tensors)].pack_into(views.buf, 0, *fields)
    return range(views.at, views.at + _VIEW * len(tensors), _VIEW)


def _device(*tensors):
    """The current device, on which every tensor has to be."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on the current CUDA device ({dev})")
    return dev


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _stream = torch._C._cuda_getCurrentRawStream  # noqa: F811  (the same handle, without a Stream object)


def _ints(t, name, n=None, dtype=_I32):
    """Pointer of a contiguous int vector (of n entries, when given)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a vector" + ("" if n is None else f" of {n} entries"))
    if t.stride(0) != 1 and t.shape[0] > 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _table(t, batch):
    """(pointer, row stride, max pages) of a block table [batch, max_pages]."""
    if t.dtype is not _I32:
        raise TypeError("block_table must be torch.int32")
    if t.dim() != 2 or t.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, max_pages]")
    n = t.shape[1]
    if n > 1 and t.stride(1) != 1:
        raise ValueError("the rows of block_table must be contiguous")
    return t.data_ptr(), (t.stride(0) if batch > 1 else n), n


def _prefix(t, n, k_pages):
    """Pointer of the table of a prefix of n keys (None: no prefix)."""
    if n <= 0:
        return None
    if t is None or t.shape[0] * k_pages.shape[2] < n:
        raise ValueError(f"prefix_table does not hold {n} keys")
    return _ints(t, "prefix_table")


def _outputs(q, out, lse, out_dtype):
    if out is None:  # in the order of q's dimensions in memory
        out = torch.empty_like(q, dtype=out_dtype)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=_F32, device=q.device)
    return out, lse


def _workspace(given, need, q):
    """(tensor or None, pointer, bytes)"""
    if given is None:
        if need == 0:
            return None, None, 0
        given = torch.empty(need, dtype=_U8, device=q.device)
    return given, given.data_ptr(), given.numel()


def page_map(block_table, ctx_lens, new_lens, free_pages, page_size, n_tokens):
    """Pages and slots of one step's new tokens, from the request lengths.

    block_table int32 [B, max_pages] is updated in place: sequence b takes
    ceil((ctx + new) / page) - ceil(ctx / page) entries of free_pages (int32), in
    order, into the next entries of its row (-1 once free_pages has run out).
    Returns (slot_map int64 [n_tokens], cu_new int32 [B + 1], kv_lens int32 [B],
    taken int32 [1]): the slots of the packed new tokens (-1 past the last one
    and where there is no page), the first token of each sequence, the lengths
    with the new tokens, and the number of pages asked for (compare it with
    len(free_pages))."""
    lib = _lib._lib or load()
    dev = _device(block_table, ctx_lens, new_lens, free_pages)
    if ctx_lens.dim() != 1:
        raise ValueError("ctx_lens must be a vector")
    batch, n_tokens = ctx_lens.shape[0], int(n_tokens)
    if n_tokens < 0:
        raise ValueError("n_tokens must not be negative")
    table, stride, width = _table(block_table, batch)
    ctx, new, free = (_ints(ctx_lens, "ctx_lens"), _ints(new_lens, "new_lens", batch),
                      _ints(free_pages, "free_pages"))
    slots = torch.empty(n_tokens, dtype=_I64, device=ctx_lens.device)
    cu = torch.empty(batch + 1, dtype=_I32, device=ctx_lens.device)
    lens = torch.empty_like(ctx_lens)
    taken = torch.empty(1, dtype=_I32, device=ctx_lens.device)
    check(lib.attn_page_map(ctx, new, batch, free, free_pages.shape[0], int(page_size), table,
                            stride, width, slots.data_ptr(), n_tokens, cu.data_ptr(),
                            lens.data_ptr(), taken.data_ptr(), _stream(dev)), "attn_page_map")
    return slots, cu, lens, taken


def page_append(k, v, k_pages, v_pages, slot_map):
    """Writes rows k, v [1, Hkv, T, D] (bf16, or f32 rounded once) into the slots
    slot_map int64 [T] of the pages; slots < 0 are skipped, the others distinct."""
    lib = _lib._lib or load()
    dev = _device(k, v, k_pages, v_pages, slot_map)
    slots = _ints(slot_map, "slot_map", k.shape[2], _I64)
    vk, vv, kp, vp = _pack(k, v, k_pages, v_pages)
    check(lib.attn_page_append(vk, vv, slots, kp, vp, _stream(dev)), "attn_page_append")


def page_append_q8(k, v, k_pages, k_scales, v_pages, v_scales, slot_map):
    """Quantises rows k, v [1, Hkv, T, D] (bf16 or f32) into the slots slot_map
    int64 [T] of an 8-bit cache; slots < 0 are skipped, the others distinct."""
    lib = _lib._lib or load()
    dev = _device(k, v, k_pages, k_scales, v_pages, v_scales, slot_map)
    slots = _ints(slot_map, "slot_map", k.shape[2], _I64)
    vk, vv, kp, ks, vp, vs = _pack(k, v, k_pages, k_scales, v_pages, v_scales, kinds=_KINDS8)
    check(lib.attn_page_append_q8(vk, vv, slots, kp, ks, vp, vs, _stream(dev)), "attn_page_append_q8")


def page_read_q8(k_pages, k_scales, v_pages, v_scales, block_table, first, cu, n_tokens, out=None,
                 out_dtype=None):
    """Rows of an 8-bit cache as numbers: positions first[b], first[b] + 1, ... of
    sequence b (int32 [B]) at the packed rows [cu[b], cu[b + 1]) (int32 [B + 1]).
    Returns (k, v) [1, Hkv, n_tokens, D], bf16 (which holds every value exactly)
    or f32, or the pair given as out; rows of no sequence are not written."""
    lib = _lib._lib or load()
    n_tokens = int(n_tokens)
    if n_tokens < 0:
        raise ValueError("n_tokens must not be negative")
    if k_pages.dim() != 4:
        raise ValueError("pages must be [P, Hkv, page, D]")
    if out is None:  # a token's heads together
        h, d = k_pages.shape[1], k_pages.shape[3]
        shape, stride = (1, h, n_tokens, d), (n_tokens * h * d, d, h * d, 1)
        out = tuple(torch.empty_strided(shape, stride, dtype=out_dtype or _BF16, device=k_pages.device)
                    for _ in range(2))
    k, v = out
    if k.shape[2] != n_tokens:
        raise ValueError(f"out must hold {n_tokens} rows")
    dev = _device(k_pages, k_scales, v_pages, v_scales, block_table, first, cu, k, v)
    batch = first.shape[0] if first.dim() == 1 else -1
    table, stride, width = _table(block_table, batch)
    at, ends = _ints(first, "first"), _ints(cu, "cu", batch + 1)
    kp, ks, vp, vs, vk, vv = _pack(k_pages, k_scales, v_pages, v_scales, k, v, kinds=_KINDS8)
    check(lib.attn_page_read_q8(kp, ks, vp, vs, table, stride, width, at, ends, batch, vk, vv,
                                _stream(dev)), "attn_page_read_q8")
    return k, v


def paged_decode(q, k_pages, v_pages, block_table, kv_lens, scale=None, prefix_table=None,
                 prefix_len=0, out=None, lse=None, workspace=None, out_dtype=None):
    """One or a few query tokens per sequence: q [B, Hq, Nq, D], the last Nq
    tokens of each sequence, (Hq / Hkv) * Nq <= 64.  With prefix_table (int32
    page numbers) every query sees prefix_len keys before its own, read once
    for many sequences together.  Returns (O, LSE)."""
    lib = _lib._lib or load()
    dev = _device(q, k_pages, v_pages, block_table, kv_lens, prefix_table, out, lse, workspace)
    out, lse = _outputs(q, out, lse, out_dtype)
    b = q.shape[0]
    table, stride, width = _table(block_table, b)
    lens = _ints(kv_lens, "kv_lens", b)
    prefix_len, prefix = int(prefix_len), _prefix(prefix_table, int(prefix_len), k_pages)
    vq, kp, vp, vo, vl = _pack(q, k_pages, v_pages, out, lse)
    ws, at, have = _workspace(
        workspace, lib.attn_paged_decode_workspace_size(vq, kp, width, prefix_len), q)
    check(lib.attn_paged_decode(vq, kp, vp, table, stride, width, lens, prefix, prefix_len,
                                -1.0 if scale is None else float(scale), vo, vl, at, have,
                                _stream(dev)), "attn_paged_decode")
    return out, lse


def paged_decode_workspace_size(q, k_pages, max_pages, prefix_len=0) -> int:
    vq, kp = _pack(q, k_pages)
    return int(load().attn_paged_decode_workspace_size(vq, kp, int(max_pages), int(prefix_len)))


def paged_fwd(q, k_pages, v_pages, block_table, kv_lens, cu_q, scale=None, out=None, lse=None,
              workspace=None, out_dtype=None):
    """Ragged prompts, causal: q [1, Hq, T, D] holds the packed tokens of every
    sequence, those of sequence b at [cu_q[b], cu_q[b + 1]) (int32 [B + 1]), the
    last tokens of its kv_lens[b].  Returns (O, LSE) of the packed tokens; rows
    of no sequence are not written."""
    lib = _lib._lib or load()
    dev = _device(q, k_pages, v_pages, block_table, kv_lens, cu_q, out, lse, workspace)
    out, lse = _outputs(q, out, lse, out_dtype)
    batch = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    table, stride, width = _table(block_table, batch)
    lens, cu = _ints(kv_lens, "kv_lens"), _ints(cu_q, "cu_q", batch + 1)
    vq, kp, vp, vo, vl = _pack(q, k_pages, v_pages, out, lse)
    ws, at, have = _workspace(
        workspace, lib.attn_paged_fwd_workspace_size(vq, kp, batch, width), q)
    check(lib.attn_paged_fwd(vq, kp, vp, table, stride, width, lens, cu, batch,
                             -1.0 if scale is None else float(scale), vo, vl, at, have,
                             _stream(dev)), "attn_paged_fwd")
    return out, lse


def paged_fwd_workspace_size(q, k_pages, batch, max_pages) -> int:
    vq, kp = _pack(q, k_pages)
    return int(load().attn_paged_fwd_workspace_size(vq, kp, int(batch), int(max_pages)))


def paged_decode_q8(q, k_pages, k_scales, v_pages, v_scales, block_table, kv_lens, scale=None,
                    prefix_table=None, prefix_len=0, out=None, lse=None, workspace=None,
                    out_dtype=None):
    """paged_decode over an 8-bit cache: attention over the numbers that it stands
    for, with P to 11 bits (out_dtype f32: 22).  Returns (O, LSE)."""
    lib = _lib._lib or load()
    dev = _device(q, k_pages, k_scales, v_pages, v_scales, block_table, kv_lens, prefix_table, out,
                  lse, workspace)
    out, lse = _outputs(q, out, lse, out_dtype)
    b = q.shape[0]
    table, stride, width = _table(block_table, b)
    lens = _ints(kv_lens, "kv_lens", b)
    prefix_len, prefix = int(prefix_len), _prefix(prefix_table, int(prefix_len), k_pages)
    vq, kp, ks, vp, vs, vo, vl = _pack(q, k_pages, k_scales, v_pages, v_scales, out, lse,
                                       kinds=_KINDS8)
    ws, at, have = _workspace(
        workspace, lib.attn_paged_decode_q8_workspace_size(vq, kp, width, prefix_len), q)
    check(lib.attn_paged_decode_q8(vq, kp, ks, vp, vs, table, stride, width, lens, prefix, prefix_len,
                                   -1.0 if scale is None else float(scale), vo, vl, at, have,
                                   _stream(dev)), "attn_paged_decode_q8")
    return out, lse


def paged_decode_q8_workspace_size(q, k_pages, max_pages, prefix_len=0) -> int:
    vq, kp = _pack(q, k_pages, kinds=_KINDS8)
    return int(load().attn_paged_decode_q8_workspace_size(vq, kp, int(max_pages), int(prefix_len)))


def paged_fwd_q8(q, k_pages, k_scales, v_pages, v_scales, block_table, kv_lens, cu_q, scale=None,
                 out=None, lse=None, workspace=None, out_dtype=None):
    """paged_fwd over an 8-bit cache: attention over the numbers that it stands for.
    Where the sequences have more than 8 D query rows of a kv head on the average, a
    bf16 copy of the pages that they see is made in the workspace, up to 4 GiB (its room
    follows from the pool and the table's width).  With a workspace of
    paged_fwd_q8_workspace_size(..., copy=False) bytes the call goes without the copy.
    Returns (O, LSE) of the packed tokens."""
    lib = _lib._lib or load()
    dev = _device(q, k_pages, k_scales, v_pages, v_scales, block_table, kv_lens, cu_q, out, lse,
                  workspace)
    out, lse = _outputs(q, out, lse, out_dtype)
    batch = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    table, stride, width = _table(block_table, batch)
    lens, cu = _ints(kv_lens, "kv_lens"), _ints(cu_q, "cu_q", batch + 1)
    vq, kp, ks, vp, vs, vo, vl = _pack(q, k_pages, k_scales, v_pages, v_scales, out, lse,
                                       kinds=_KINDS8)
    ws, at, have = _workspace(
        workspace, lib.attn_paged_fwd_q8_workspace_size(vq, kp, batch, width), q)
    check(lib.attn_paged_fwd_q8(vq, kp, ks, vp, vs, table, stride, width, lens, cu, batch,
                                -1.0 if scale is None else float(scale), vo, vl, at, have,
                                _stream(dev)), "attn_paged_fwd_q8")
    return out, lse


def paged_fwd_q8_workspace_size(q, k_pages, batch, max_pages, copy=True) -> int:
    """Bytes with room for the bf16 copy, where the sizes are for one, or (copy=False)
    without, which is enough.  A size that includes a copy can exceed that of more
    sequences or a wider table; one without it does not."""
    vq, kp = _pack(q, k_pages, kinds=_KINDS8)
    size = load().attn_paged_fwd_q8_workspace_size if copy else load().attn_paged_fwd_workspace_size
    return int(size(vq, kp, int(batch), int(max_pages)))
