"""Plain forms of the paged operators for the tests: pages as Python lists,
attention by the fp64 oracle on each sequence's gathered keys."""

import numpy as np
import torch

from helpers import f64
from oracle import attention as A

U16 = 2.0 ** -8   # half a step of bf16, relative
U32 = 2.0 ** -24  # half a step of fp32


def page_map(table, ctx, new, free, page, n_tokens):
    """(table, slots, cu, lens, taken) token by token."""
    table = [list(r) for r in table]
    ctx, new = [max(0, c) for c in ctx], [max(0, n) for n in new]
    slots, cu, used = [], [0], 0
    for row, c, n in zip(table, ctx, new):
        for pos in range(c, c + n):
            at = pos // page
            if pos % page == 0:
                if at < len(row):
                    row[at] = free[used] if used < len(free) else -1
                used += 1
            slots.append(row[at] * page + pos % page if at < len(row) and row[at] >= 0 else -1)
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * max(0, n_tokens - len(slots)))[:n_tokens]
    return table, slots, cu, [c + n for c, n in zip(ctx, new)], used


def keys_of(pages, row, n):
    """Rows 0..n-1 of the sequence with pages `row`: [Hkv, n, D] fp64, and which of
    them exist (a page number outside the pool has no rows)."""
    page = pages.shape[2]
    numbers = [int(x) for x in row[: -(-n // page)]]
    ok = np.repeat([0 <= g < pages.shape[0] for g in numbers], page)[:n].astype(bool)
    idx = torch.tensor([g if 0 <= g < pages.shape[0] else 0 for g in numbers], dtype=torch.long,
                       device=pages.device)
    rows = f64(pages[idx].transpose(0, 1).flatten(1, 2)[:, :n]) if n else np.zeros((pages.shape[1], 0, pages.shape[3]))
    return rows, ok


def attend(q, k, v, last, ok, scale=None):
    """q [Hq, R, D], k, v [Hkv, N, D]; row r sees keys j <= last[r] with ok[j]."""
    hq, r, d = q.shape
    o, lse = np.zeros((hq, r, d)), np.full((hq, r), -np.inf)
    for i in range(r):
        see = ok.copy()
        see[max(0, last[i] + 1):] = False
        if see.any():
            oo, ll = A.attn_fwd(q[None, :, i:i + 1], k[None][:, :, see], v[None][:, :, see], scale=scale)
            o[:, i], lse[:, i] = oo[0, :, 0], ll[0, :, 0]
    return o, lse


def decode(q, kp, vp, table, lens, prefix=(), prefix_len=0, scale=None):
    Q, out, lses = f64(q), [], []
    nq, cap = q.shape[2], table.shape[1] * kp.shape[2]
    tab = table.cpu().tolist()
    pk, pok = keys_of(kp, prefix, prefix_len)
    pv, _ = keys_of(vp, prefix, prefix_len)
    for b, n in enumerate(lens):
        full, n = n, min(max(n, 0), cap)
        k, ok = keys_of(kp, tab[b], n)
        v, _ = keys_of(vp, tab[b], n)
        last = [max(min(full - nq + i, n - 1), -1) + prefix_len for i in range(nq)]
        o, l_ = attend(Q[b], np.concatenate([pk, k], 1), np.concatenate([pv, v], 1), last,
                       np.concatenate([pok, ok]), scale)
        out.append(o)
        lses.append(l_)
    return np.stack(out), np.stack(lses)


def fwd(q, kp, vp, table, lens, cu, scale=None):
    """Rows of no sequence stay NaN."""
    Q = f64(q)[0]
    o, lse = np.full(Q.shape, np.nan), np.full(Q.shape[:2], np.nan)
    tab = table.cpu().tolist()
    for b, n in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        k, ok = keys_of(kp, tab[b], n)
        v, _ = keys_of(vp, tab[b], n)
        last = [n - (cu[b + 1] - cu[b]) + i for i in range(cu[b + 1] - cu[b])]
        if ok.all() and n >= cu[b + 1] - cu[b] > 0:  # the whole sequence at once
            oo, ll = A.attn_fwd(Q[None, :, rows], k[None], v[None], last[0], 0, True, scale)
            o[:, rows], lse[:, rows] = oo[0], ll[0]
        else:
            o[:, rows], lse[:, rows] = attend(Q[:, rows], k, v, last, ok, scale)
    return o[None], lse[None]


def score_error(q, k, scale=None):
    """How far a score may be off: D products (exact in fp32) are added and
    scaled in fp32, each step within half a step of the running sum of absolute
    values: (D + 2) * 2^-24 * scale * max |q|_2 |k|_2.  The tensor cores add
    with truncation instead of rounding, a whole step: twice that."""
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    big = float(q.float().norm(dim=-1).max()) * float(k.float().norm(dim=-1).max())
    return 2 * (d + 2) * U32 * scale * big


def tolerances(q, kp, vp, p_rounding, out_dtype, scale=None):
    """(O, LSE) bounds.  A weight p_j = exp2(s_j - m) is off by e_s (its score),
    2^-19 (the fp32 argument, below 2^5: half a step of it) and 2^-21 (the
    exponential), and by p_rounding relative in the numerator; fp32 sums add a few
    2^-24 * sqrt(n) (taken as 2^-19): |dO| <= (2 (..) + p_rounding) max|v|, and a
    bf16 output half a step of |O| <= max|v|.  |dLSE| <= those, plus fp32 rounding
    of an LSE below 64 (2^-19)."""
    es = score_error(q, kp, scale)
    vmax = float(vp.float().abs().max())
    rel = es + 2.0 ** -19 + 2.0 ** -21 + 2.0 ** -19
    tol = (2 * rel + p_rounding) * vmax
    if out_dtype == torch.bfloat16:
        tol += U16 * vmax
    return tol, rel + 2.0 ** -19
