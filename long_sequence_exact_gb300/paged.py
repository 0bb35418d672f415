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

Tensors live on the current CUDA device; calls are enqueued on the current
stream.  Inference only: no gradients are recorded.  A page number, slot or
length outside the cache is skipped on the device and reported by
``sync_status`` (LSX_ERR_PAGE).
"""

from __future__ import annotations

from ctypes import byref

import torch

from ._lib import check, load, stream_handle, view

_I32, _I64 = torch.int32, torch.int64


def _on_device(*tensors):
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on the current CUDA device ({dev})")


def _ints(t, name, n=None, dtype=_I32):
    """A contiguous int vector (of n entries, when given)."""
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
    lib = load()
    _on_device(block_table, ctx_lens, new_lens, free_pages)
    if ctx_lens.dim() != 1:
        raise ValueError("ctx_lens must be a vector")
    batch, n_tokens = ctx_lens.shape[0], int(n_tokens)
    if n_tokens < 0:
        raise ValueError("n_tokens must not be negative")
    table, stride, width = _table(block_table, batch)
    ctx, new, free = (_ints(ctx_lens, "ctx_lens"), _ints(new_lens, "new_lens", batch),
                      _ints(free_pages, "free_pages"))
    slots = block_table.new_empty(n_tokens, dtype=_I64)
    cu, lens, taken = ctx_lens.new_empty(2 * batch + 2).split((batch + 1, batch, 1))
    check(lib.attn_page_map(ctx, new, batch, free, free_pages.shape[0], int(page_size), table,
                            stride, width, slots.data_ptr(), n_tokens, cu.data_ptr(),
                            lens.data_ptr(), taken.data_ptr(), stream_handle()), "attn_page_map")
    return slots, cu, lens, taken


def page_append(k, v, k_pages, v_pages, slot_map):
    """Writes rows k, v [1, Hkv, T, D] (bf16, or f32 rounded once) into the slots
    slot_map int64 [T] of the pages; slots < 0 are skipped, the others distinct."""
    lib = load()
    _on_device(k, v, k_pages, v_pages, slot_map)
    vk, vv, kp, vp = view(k), view(v), view(k_pages), view(v_pages)
    slots = _ints(slot_map, "slot_map", k.shape[2], _I64)
    check(lib.attn_page_append(byref(vk), byref(vv), slots, byref(kp), byref(vp),
                               stream_handle()), "attn_page_append")


def paged_decode(q, k_pages, v_pages, block_table, kv_lens, scale=None, prefix_table=None,
                 prefix_len=0, out=None, lse=None, workspace=None, out_dtype=None):
    """One or a few query tokens per sequence: q [B, Hq, Nq, D], the last Nq
    tokens of each sequence, (Hq / Hkv) * Nq <= 64.  With prefix_table (int32
    page numbers) every query sees prefix_len keys before its own, read once
    for many sequences together.  Returns (O, LSE)."""
    lib = load()
    b, h, n, d = q.shape
    _on_device(q, k_pages, v_pages, block_table, kv_lens, prefix_table, out, lse, workspace)
    if out is None:
        out = q.new_empty((b, h, n, d), dtype=out_dtype or q.dtype)
    if lse is None:
        lse = q.new_empty((b, h, n), dtype=torch.float32)
    table, stride, width = _table(block_table, b)
    lens = _ints(kv_lens, "kv_lens", b)
    prefix_len, prefix = int(prefix_len), None
    if prefix_len > 0:
        if prefix_table is None or prefix_table.shape[0] * k_pages.shape[2] < prefix_len:
            raise ValueError(f"prefix_table does not hold {prefix_len} keys")
        prefix = _ints(prefix_table, "prefix_table")
    vq, kp, vp, vo, vl = view(q), view(k_pages), view(v_pages), view(out), view(lse)
    if workspace is None:
        workspace = q.new_empty(lib.attn_paged_decode_workspace_size(
            byref(vq), byref(kp), width, prefix_len), dtype=torch.uint8)
    check(lib.attn_paged_decode(byref(vq), byref(kp), byref(vp), table, stride, width, lens,
                                prefix, prefix_len, -1.0 if scale is None else float(scale),
                                byref(vo), byref(vl), workspace.data_ptr(), workspace.numel(),
                                stream_handle()), "attn_paged_decode")
    return out, lse


def paged_decode_workspace_size(q, k_pages, max_pages, prefix_len=0) -> int:
    vq, kp = view(q), view(k_pages)
    return int(load().attn_paged_decode_workspace_size(byref(vq), byref(kp), int(max_pages),
                                                       int(prefix_len)))


def paged_fwd(q, k_pages, v_pages, block_table, kv_lens, cu_q, scale=None, out=None, lse=None,
              workspace=None, out_dtype=None):
    """Ragged prompts, causal: q [1, Hq, T, D] holds the packed tokens of every
    sequence, those of sequence b at [cu_q[b], cu_q[b + 1]) (int32 [B + 1]), the
    last tokens of its kv_lens[b].  Returns (O, LSE) of the packed tokens; rows
    of no sequence are not written."""
    lib = load()
    b, h, n, d = q.shape
    _on_device(q, k_pages, v_pages, block_table, kv_lens, cu_q, out, lse, workspace)
    if out is None:
        out = q.new_empty((b, h, n, d), dtype=out_dtype or q.dtype)
    if lse is None:
        lse = q.new_empty((b, h, n), dtype=torch.float32)
    batch = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    table, stride, width = _table(block_table, batch)
    lens, cu = _ints(kv_lens, "kv_lens"), _ints(cu_q, "cu_q", batch + 1)
    vq, kp, vp, vo, vl = view(q), view(k_pages), view(v_pages), view(out), view(lse)
    if workspace is None:
        workspace = q.new_empty(lib.attn_paged_fwd_workspace_size(
            byref(vq), byref(kp), batch, width), dtype=torch.uint8)
    check(lib.attn_paged_fwd(byref(vq), byref(kp), byref(vp), table, stride, width, lens, cu,
                             batch, -1.0 if scale is None else float(scale), byref(vo), byref(vl),
                             workspace.data_ptr(), workspace.numel(), stream_handle()),
          "attn_paged_fwd")
    return out, lse


def paged_fwd_workspace_size(q, k_pages, batch, max_pages) -> int:
    vq, kp = view(q), view(k_pages)
    return int(load().attn_paged_fwd_workspace_size(byref(vq), byref(kp), int(batch),
                                                    int(max_pages)))
