"""The paged cache against plain forms: page maps (exact integers), cache
writes (bit for bit), paged decode and paged prompts (the fp64 oracle on each
sequence's gathered keys)."""

import numpy as np
import pytest
import torch

import long_sequence_exact_gb300 as lsx
import paged_ref as P
from helpers import check_close, check_lse, f64
from long_sequence_exact_gb300.inputs import random_tensor

pytestmark = pytest.mark.gpu
DEV = "cuda"
P_SPLIT = 2.0 ** -16   # decode: P as a sum of two bf16
P_BF16 = 2.0 ** -8     # prompts, and a prefix under more than 32 query rows: P rounded to bf16


def p_rounding(q, kp, prefix_len):
    rows = q.shape[0] * (q.shape[1] // kp.shape[1]) * q.shape[2]
    return P_BF16 if prefix_len and rows > 32 else P_SPLIT


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def pool(n, hkv, page, d, seed, token_major=True):
    if token_major:
        return random_tensor((n, page, hkv, d), seed, device=DEV).transpose(1, 2)
    return random_tensor((n, hkv, page, d), seed, device=DEV)


def tables(lens, page, n_pages, seed, width=None, fill=-1):
    need = [-(-max(n, 0) // page) for n in lens]
    order = np.random.default_rng(seed).permutation(n_pages)
    t = np.full((len(lens), max([width or 1] + need)), fill, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t).to(DEV), [int(x) for x in order[at:]]


def poison(kp, vp, table, lens, page, prefix=(), prefix_len=0):
    """NaN into every row that no sequence holds."""
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    tab = table.cpu().tolist()
    for row, n in [(r, m) for r, m in zip(tab, lens)] + [(list(prefix), prefix_len)]:
        for i in range(n):
            used[row[i // page], i % page] = True
    dead = ~used.to(DEV)[:, None, :, None]
    for x in (kp, vp):
        x.masked_fill_(dead, float("nan"))


def done():
    torch.cuda.synchronize()
    return lsx.sync_status()


# ------------------------------------------------------------------ page maps
@pytest.mark.parametrize("batch,page,ctx_max,new_max", [
    (1, 16, 0, 1), (1, 256, 700, 1), (3, 16, 0, 50), (64, 16, 500, 1), (257, 32, 300, 3),
    (1000, 64, 900, 70), (4096, 16, 100, 2), (5, 128, 3000, 20000),
])
@pytest.mark.parametrize("short", [0, 3])
def test_page_map(batch, page, ctx_max, new_max, short):
    r = np.random.default_rng(batch + page)
    ctx = r.integers(0, ctx_max + 1, batch)
    new = r.integers(0, new_max + 1, batch)
    new[0], ctx[batch // 2] = new_max, 0
    if batch > 2:
        ctx[1], new[1] = -7, -5    # negative lengths count as none
        new[2] = 0
    need = int(np.sum(-(-(np.maximum(ctx, 0) + np.maximum(new, 0)) // page) - -(-np.maximum(ctx, 0) // page)))
    n_pages = 3 * batch + 2 * need + int(np.sum(np.maximum(ctx, 0) // page)) + 9
    width = max(1, int((np.maximum(ctx, 0) + np.maximum(new, 0)).max()) // page + 1 - short)
    order = [int(x) for x in r.permutation(n_pages)]
    free = order[: max(0, need - short)]
    table = r.integers(0, n_pages, (batch, width + 3)).astype(np.int32)
    table[:, width - 1] = -1
    tokens = int(np.maximum(new, 0).sum()) + (5 if short == 0 else -1)
    tokens = max(tokens, 0)
    ref = P.page_map(table[:, :width].tolist(), ctx.tolist(), new.tolist(), free, page, tokens)
    whole = torch.from_numpy(table).to(DEV)
    for _ in range(2):  # the same again on the updated table
        slots, cu, lens, taken = lsx.page_map(whole[:, :width], ints(ctx), ints(new), ints(free), page, tokens)
        assert done() == 0
        got = whole.cpu().numpy()
        assert np.array_equal(got[:, width:], table[:, width:])
        assert got[:, :width].tolist() == ref[0]
        assert slots.cpu().tolist() == ref[1]
        assert cu.cpu().tolist() == ref[2]
        assert lens.cpu().tolist() == ref[3]
        assert taken.cpu().tolist() == [ref[4]]


@pytest.mark.parametrize("ctx,new", [
    ([2 ** 31 - 1, 5, -2 ** 31], [1, 2 ** 31 - 1, 2 ** 31 - 1]), ([2 ** 31 - 1] * 3, [2 ** 31 - 1] * 3),
    ([0] * 5, [2 ** 31 - 1] * 5),
])
def test_page_map_with_sums_past_31_bits_stays_inside_its_arrays(ctx, new):
    """What such lengths give is not defined; nothing outside the outputs changes."""
    b = len(ctx)
    whole = torch.full((b + 2, 9), 77, dtype=torch.int32, device=DEV)
    free = ints([3, 4, 5])
    slots, cu, lens, taken = lsx.page_map(whole[1:-1, 2:6], ints(ctx), ints(new), free, 16, 50)
    assert done() == 0
    assert whole[0].eq(77).all() and whole[-1].eq(77).all()
    assert whole[:, :2].eq(77).all() and whole[:, 6:].eq(77).all()
    assert (slots < 16 * 78).all() and free.tolist() == [3, 4, 5]


def test_page_map_without_tokens_or_pages():
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    slots, cu, lens, taken = lsx.page_map(table, ints([0, 5]), ints([0, 0]), ints([]), 16, 0)
    assert done() == 0
    assert slots.numel() == 0 and cu.tolist() == [0, 0, 0] and lens.tolist() == [0, 5] and taken.tolist() == [0]
    slots, cu, lens, taken = lsx.page_map(table, ints([0, 16]), ints([2, 1]), ints([]), 16, 4)
    assert done() == 0
    assert slots.tolist() == [-1] * 4 and taken.tolist() == [2] and table.eq(-1).all()


# --------------------------------------------------------------------- writes
@pytest.mark.parametrize("tokens,hkv,d,page,token_major,dtype", [
    (1, 1, 64, 16, True, torch.bfloat16), (64, 8, 128, 16, True, torch.bfloat16),
    (333, 3, 128, 64, False, torch.bfloat16), (1001, 2, 64, 256, True, torch.float32),
    (77, 5, 128, 32, False, torch.float32),
])
def test_page_append(tokens, hkv, d, page, token_major, dtype):
    n = -(-tokens // page) + 2
    kp, vp = pool(n, hkv, page, d, 1, token_major), pool(n, hkv, page, d, 2, token_major)
    # rows inside a wider projection: token stride larger than Hkv * D
    wide = random_tensor((tokens, hkv + 1, 2 * d), 3, dtype=dtype, device=DEV)
    k = wide[:, :hkv, :d].transpose(0, 1)[None]
    v = wide[:, 1:, d:].transpose(0, 1)[None]
    slots = np.random.default_rng(4).permutation(n * page)[:tokens].astype(np.int64)
    slots[1::5] = -1
    want_k, want_v = kp.clone(), vp.clone()
    for t, s in enumerate(slots):
        if s >= 0:
            want_k[s // page, :, s % page] = k[0, :, t].to(torch.bfloat16)
            want_v[s // page, :, s % page] = v[0, :, t].to(torch.bfloat16)
    lsx.page_append(k, v, kp, vp, ints(slots, torch.int64))
    assert done() == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_page_append_skips_a_slot_past_the_pool():
    kp, vp = pool(2, 2, 16, 64, 1), pool(2, 2, 16, 64, 2)
    k = random_tensor((1, 2, 3, 64), 3, device=DEV)
    want = kp.clone()
    want[0, :, 5] = k[0, :, 1]
    lsx.page_append(k, k, kp, vp, ints([32, 5, 1 << 40], torch.int64))
    assert done() == -10
    assert torch.equal(kp, want)
    assert done() == 0


# --------------------------------------------------------------------- decode
DECODE = [
    # Hq, Hkv, Nq, D, page, lens, prefix
    (1, 1, 1, 64, 16, [1], 0),
    (4, 1, 1, 128, 16, [0, 1, 15, 16, 17, 33, 64, 65], 0),
    (8, 2, 1, 128, 32, [700, 0, 1300, 5], 0),
    (2, 2, 1, 64, 64, [129, 2000, 63], 0),
    (16, 1, 1, 128, 16, [300, 301], 0),
    (40, 2, 1, 64, 256, [513, 255, 256, 257], 0),        # 20 rows a key head
    (64, 1, 1, 128, 64, [190, 1000], 0),                 # 64 rows
    (6, 2, 3, 128, 16, [2, 3, 40, 0, 1, 129], 0),        # fewer keys than query tokens: rows without keys
    (8, 8, 5, 64, 128, [1000, 4, 5, 6], 0),
    (5, 1, 12, 128, 16, [12, 77], 0),                    # 60 rows
    (8, 2, 1, 128, 16, [30, 0, 7, 100], 333),
    (4, 4, 1, 64, 64, [0, 0, 0], 64),                    # a prefix alone
    (4, 2, 2, 128, 32, [1, 2, 50, 300, 0, 33, 9], 1000),
    (64, 2, 1, 64, 16, [100, 20], 500),
    (3, 3, 1, 128, 16, [10] * 70, 257),                  # more branches than one group of rows
    (8, 1, 1, 128, 64, [40 * i for i in range(20)], 4096),
    (2, 1, 1, 128, 128, [30011], 0),                     # one long sequence, many splits
]


def decode_case(hq, hkv, nq, d, page, lens, prefix_len, seed=50, token_major=True, width=None):
    need = sum(-(-n // page) for n in lens) + -(-prefix_len // page)
    n_pages = need + 3
    kp, vp = pool(n_pages, hkv, page, d, seed, token_major), pool(n_pages, hkv, page, d, seed + 1, token_major)
    table, rest = tables(lens, page, n_pages, seed, width)
    prefix = rest[: -(-prefix_len // page)]
    q = random_tensor((len(lens), nq, hq, d), seed + 2, device=DEV).transpose(1, 2)
    return q, kp, vp, table, prefix


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c[:5])) + f"-{len(c[5])}-{c[6]}")
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("keys", [0, 40000])  # what the table can hold: narrow tables take clusters
def test_paged_decode(case, out_dtype, keys):
    hq, hkv, nq, d, page, lens, prefix_len = case
    q, kp, vp, table, prefix = decode_case(*case, token_major=out_dtype is torch.float32, width=keys // page)
    tol, tol_lse = P.tolerances(q, kp, vp, p_rounding(q, kp, prefix_len), out_dtype)
    o_ref, l_ref = P.decode(q, kp, vp, table, lens, prefix, prefix_len)
    poison(kp, vp, table, lens, page, prefix, prefix_len)
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), prefix_table=ints(prefix) if prefix_len else None,
                              prefix_len=prefix_len, out_dtype=out_dtype)
    assert done() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)


@pytest.mark.parametrize("i", range(24))
def test_paged_decode_random(i):
    r = np.random.default_rng(7000 + i)
    hkv = int(r.integers(1, 5))
    g = int(r.choice([1, 2, 3, 4, 7, 8, 16]))
    nq = int(r.integers(1, 64 // g + 1)) if r.random() < 0.4 else 1
    d, page = int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128, 256]))
    lens = [int(x) for x in r.integers(0, int(r.choice([20, 300, 2500])), int(r.integers(1, 12)))]
    prefix_len = int(r.integers(1, 1500)) if r.random() < 0.4 else 0
    q, kp, vp, table, prefix = decode_case(hkv * g, hkv, nq, d, page, lens, prefix_len, 90 + i,
                                           bool(r.integers(0, 2)), int(r.choice([1, 40000 // page])))
    scale = float(r.choice([0.05, 0.125, 0.3]))
    tol, tol_lse = P.tolerances(q, kp, vp, p_rounding(q, kp, prefix_len), torch.float32, scale)
    o_ref, l_ref = P.decode(q, kp, vp, table, lens, prefix, prefix_len, scale)
    poison(kp, vp, table, lens, page, prefix, prefix_len)
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), scale, ints(prefix) if prefix_len else None,
                              prefix_len, out_dtype=torch.float32)
    assert done() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)


def test_paged_decode_leaves_out_pages_that_do_not_exist():
    case = (8, 2, 2, 128, 16, [100, 40, 90, 16], 70)
    hq, hkv, nq, d, page, lens, prefix_len = case
    q, kp, vp, table, prefix = decode_case(*case)
    table[0, 2], table[1, 0], table[2, 5] = -1, kp.shape[0], 2 ** 31 - 1
    table[3, 0] = -2 ** 31                    # all keys of the last sequence
    prefix[1] = -5
    o_ref, l_ref = P.decode(q, kp, vp, table, lens, prefix, prefix_len)
    tol, tol_lse = P.tolerances(q, kp, vp, P_SPLIT, torch.float32)
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), prefix_table=ints(prefix), prefix_len=prefix_len,
                              out_dtype=torch.float32)
    assert done() == -10
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)
    assert done() == 0


def test_paged_decode_lengths_outside_the_table():
    case = (4, 2, 2, 64, 16, [64, 64, 64], 0)
    q, kp, vp, table, _ = decode_case(*case)
    tol, tol_lse = P.tolerances(q, kp, vp, P_SPLIT, torch.float32)
    # 64 keys fit a row of the table
    for lens, status in (([-3, 20, 64], 0), ([5000, 65, 66], -10), ([2 ** 31 - 1, -2 ** 31, 1], -10)):
        o_ref, l_ref = P.decode(q, kp, vp, table, lens)
        o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), out_dtype=torch.float32)
        assert done() == status
        check_lse(f64(lse), l_ref, tol_lse)
        check_close(f64(o), o_ref, tol)


def test_paged_decode_writes_only_its_rows():
    q, kp, vp, table, _ = decode_case(4, 2, 1, 128, 16, [40, 0, 3], 0)
    big = torch.full((3, 4, 3, 128 + 64), 7.0, device=DEV)
    lbig = torch.full((3, 4, 3), 7.0, device=DEV)
    out, lse = big[:, :, 1:2, :128], lbig[:, :, 1:2]
    o2, l2 = lsx.paged_decode(q, kp, vp, table, ints([40, 0, 3]), out=out, lse=lse)
    assert done() == 0 and o2 is out and l2 is lse
    o3, l3 = lsx.paged_decode(q, kp, vp, table, ints([40, 0, 3]), out_dtype=torch.float32)
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    out.fill_(7.0)
    lse.fill_(7.0)
    assert big.eq(7.0).all() and lbig.eq(7.0).all()


def test_paged_decode_is_bit_repeatable_and_takes_any_workspace():
    case = (8, 2, 1, 128, 16, [2500, 10, 900, 0, 77], 3000)
    q, kp, vp, table, prefix = decode_case(*case)
    args = (q, kp, vp, table, ints(case[5]), None, ints(prefix), 3000)
    need = lsx.paged_decode_workspace_size(q, kp, table.shape[1], 3000)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((max(need, 1) + 256,), fill, dtype=torch.uint8, device=DEV)
        ws = ws[(-ws.data_ptr()) % 256:]
        outs.append(lsx.paged_decode(*args, workspace=ws))
    assert done() == 0
    for o, l_ in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l_, outs[0][1])


def test_paged_decode_far_offsets():
    """Pages past 2^31 elements and 2^32 bytes of the pool."""
    hkv, page, d = 8, 256, 128
    n_pages = 2 ** 33 // (hkv * page * d * 2) + 40   # a little over 8 GiB each
    kp = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    vp = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    use = [n_pages - 1, 0, n_pages // 2 + 1, n_pages - 2]
    for i, g in enumerate(use):
        kp[g] = random_tensor((hkv, page, d), 5 + i, device=DEV)
        vp[g] = random_tensor((hkv, page, d), 15 + i, device=DEV)
    small_k, small_v = kp[use].clone(), vp[use].clone()
    q = random_tensor((1, 16, 1, d), 3, device=DEV)
    lens = ints([1000])
    o, lse = lsx.paged_decode(q, kp, vp, ints([use]), lens)
    o2, lse2 = lsx.paged_decode(q, small_k, small_v, ints([[0, 1, 2, 3]]), lens)
    qq = random_tensor((1, 16, 300, d), 4, device=DEV)
    cu = ints([0, 300])
    o3, lse3 = lsx.paged_fwd(qq, kp, vp, ints([use]), lens, cu)
    o4, lse4 = lsx.paged_fwd(qq, small_k, small_v, ints([[0, 1, 2, 3]]), lens, cu)
    row = random_tensor((1, hkv, 1, d), 9, device=DEV)
    lsx.page_append(row, row, kp, vp, ints([n_pages * page - 1], torch.int64))
    assert done() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(o3, o4) and torch.equal(lse3, lse4)
    assert torch.equal(kp[n_pages - 1, :, page - 1], row[0, :, 0])


# -------------------------------------------------------------------- prompts
PROMPT = [
    # Hq, Hkv, D, page, (ctx, new) of each sequence
    (1, 1, 64, 16, [(0, 1)]),
    (4, 1, 128, 16, [(0, 5), (0, 0), (3, 1), (16, 16), (15, 18)]),
    (8, 2, 128, 32, [(0, 300), (100, 7), (0, 64)]),
    (2, 2, 64, 64, [(63, 130), (0, 257)]),
    (6, 2, 128, 128, [(0, 200), (500, 33)]),              # three heads a key head
    (5, 1, 64, 256, [(255, 40), (256, 256), (0, 1)]),
    (16, 1, 128, 16, [(40, 50)]),
    (128, 1, 64, 64, [(70, 5), (0, 9)]),                  # 128 heads: one token a row tile
    (40, 1, 128, 16, [(33, 21)]),
    (8, 8, 128, 64, [(0, 600)]),
    (4, 2, 64, 16, [(3000, 20), (0, 20)]),                # few rows, many keys
    (4, 1, 128, 64, [(i, i + 1) for i in range(40)]),
]


def prompt_case(hq, hkv, d, page, seqs, seed=60, token_major=True, tail=0):
    lens, cu = [c + n for c, n in seqs], [0]
    for _, n in seqs:
        cu.append(cu[-1] + n)
    n_pages = sum(-(-n // page) for n in lens) + 3
    kp, vp = pool(n_pages, hkv, page, d, seed, token_major), pool(n_pages, hkv, page, d, seed + 1, token_major)
    table, _ = tables(lens, page, n_pages, seed)
    q = random_tensor((cu[-1] + tail, hq, d), seed + 2, device=DEV).transpose(0, 1)[None]
    return q, kp, vp, table, lens, cu


def check_prompt(o, lse, o_ref, l_ref, tol, tol_lse):
    """Rows that no sequence has are NaN in the reference and untouched (7) here."""
    o, lse = f64(o), f64(lse)
    none = np.isnan(l_ref)
    assert (lse[none] == 7.0).all() and (o[none] == 7.0).all()
    check_lse(lse[~none], l_ref[~none], tol_lse)
    check_close(o[~none], o_ref[~none], tol)


@pytest.mark.parametrize("case", PROMPT, ids=lambda c: "-".join(map(str, c[:4])) + f"-{len(c[4])}")
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_paged_fwd(case, out_dtype):
    q, kp, vp, table, lens, cu = prompt_case(*case, token_major=out_dtype is torch.bfloat16, tail=3)
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, out_dtype)
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu)
    poison(kp, vp, table, lens, case[3])
    out = torch.full(q.shape, 7.0, dtype=out_dtype, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), out=out, lse=lse)
    assert done() == 0
    check_prompt(out, lse, o_ref, l_ref, tol, tol_lse)


@pytest.mark.parametrize("i", range(16))
def test_paged_fwd_random(i):
    r = np.random.default_rng(8000 + i)
    hkv = int(r.integers(1, 4))
    g = int(r.choice([1, 2, 3, 4, 8, 11]))
    d, page = int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128, 256]))
    seqs = [(int(r.integers(0, 900)) * int(r.integers(0, 2)), int(r.integers(0, 260))) for _ in range(int(r.integers(1, 6)))]
    q, kp, vp, table, lens, cu = prompt_case(hkv * g, hkv, d, page, seqs, 300 + i, bool(r.integers(0, 2)), 1)
    scale = float(r.choice([0.05, 0.125, 0.3]))
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.bfloat16, scale)
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu, scale)
    poison(kp, vp, table, lens, page)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), scale, out, lse)
    assert done() == 0
    check_prompt(out, lse, o_ref, l_ref, tol, tol_lse)


@pytest.mark.parametrize("case", [
    (1, 1, 128, 16, [(9000, 3)]),                             # one unit in more than eight pieces
    (2, 1, 64, 32, [(2500, 130), (0, 0), (1200, 5)]),         # cut and whole units
    (3, 3, 128, 64, [(1100 * (i % 2), 2) for i in range(20)]),
    (1, 1, 64, 16, [(i % 7, i % 2) for i in range(1100)]),    # more units than are cut, and empty ones
    (1, 1, 64, 16, [(1500, 1) if i % 200 == 7 else (5, 0) for i in range(1000)]),
], ids=["nine", "mixed", "heads", "many", "few"])
def test_paged_fwd_cut_units(case):
    """Long keys over few tokens: pieces and their merge; with outputs that are
    aligned to 16 bytes only."""
    q, kp, vp, table, lens, cu = prompt_case(*case, tail=2)
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu)
    bounds = {t: P.tolerances(q, kp, vp, P_BF16, t) for t in (torch.float32, torch.bfloat16)}
    poison(kp, vp, table, lens, case[3])
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    for dtype, shift in ((torch.float32, 0), (torch.float32, 4), (torch.bfloat16, 0), (torch.bfloat16, 8)):
        tol, tol_lse = bounds[dtype]
        flat = torch.full((q.numel() + 8,), 7.0, dtype=dtype, device=DEV)
        out = flat[shift:shift + q.numel()].view(q.shape)
        assert out.data_ptr() % 32 == (16 if shift else 0)
        lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), out=out, lse=lse)
        assert done() == 0
        check_prompt(out, lse, o_ref, l_ref, tol, tol_lse)


def check_nan_rows(o, lse, o_ref, l_ref, sees, tol, tol_lse):
    """NaN in the rows that see the NaN score, the reference elsewhere."""
    o, lse = f64(o), f64(lse)
    assert np.isnan(lse[sees]).all() and np.isnan(o[sees]).all()
    check_lse(lse[~sees], l_ref[~sees], tol_lse)
    check_close(o[~sees], o_ref[~sees], tol)


@pytest.mark.parametrize("seq", [(100, 300), (3000, 40)])  # whole; cut into pieces
@pytest.mark.parametrize("d", [64, 128])
def test_paged_fwd_nan_scores(seq, d):
    q, kp, vp, table, lens, cu = prompt_case(4, 2, d, 16, [seq, (0, 50)])
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.float32)
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu)
    at, bad = seq[0] + 20, seq[1] + 7                 # a key of the first sequence, a token of the second
    kp[int(table[0, at // 16]), 0, at % 16, 3] = float("nan")
    q[0, 3, bad] = float("nan")
    sees = np.zeros(l_ref.shape, bool)
    sees[0, :2, 20:seq[1]] = True
    sees[0, 3, bad] = True
    o, lse = lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), out_dtype=torch.float32)
    assert done() == 0
    check_nan_rows(o, lse, o_ref, l_ref, sees, tol, tol_lse)


@pytest.mark.parametrize("lens,prefix_len,keys", [
    ([700, 40], 0, 0),                 # a cluster each
    ([700, 40], 0, 40000),             # runs
    ([9000, 40], 0, 40000),            # a unit in many runs
    ([700, 40], 300, 0),               # behind a prefix, few rows
    ([700, 40] + [5] * 20, 300, 0),    # behind a prefix, many
])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_decode_nan_scores(lens, prefix_len, keys, d):
    q, kp, vp, table, prefix = decode_case(4, 2, 2, d, 16, lens, prefix_len, width=keys // 16)
    tol, tol_lse = P.tolerances(q, kp, vp, p_rounding(q, kp, prefix_len), torch.float32)
    o_ref, l_ref = P.decode(q, kp, vp, table, lens, prefix, prefix_len)
    at = lens[0] - 1                                  # the last key: of the last query token alone
    kp[int(table[0, at // 16]), 0, at % 16, 3] = float("nan")
    q[1, 3, 0] = float("nan")
    sees = np.zeros(l_ref.shape, bool)
    sees[0, :2, 1] = True
    sees[1, 3, 0] = True
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), prefix_table=ints(prefix) if prefix_len else None,
                              prefix_len=prefix_len, out_dtype=torch.float32)
    assert done() == 0
    check_nan_rows(o, lse, o_ref, l_ref, sees, tol, tol_lse)


def test_paged_fwd_leaves_out_pages_that_do_not_exist():
    q, kp, vp, table, lens, cu = prompt_case(4, 2, 128, 16, [(100, 60), (0, 33), (0, 16)])
    table[0, 1], table[0, 7], table[1, 1] = -1, kp.shape[0], 2 ** 31 - 1
    table[2, 0] = -9                          # every key of the last sequence
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.float32)
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu)
    o, lse = lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), out_dtype=torch.float32)
    assert done() == -10
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)
    assert done() == 0


def test_paged_fwd_fewer_keys_than_tokens():
    """The first tokens of such a sequence see nothing: O = 0, LSE = -inf."""
    q, kp, vp, table, _, cu = prompt_case(4, 2, 64, 16, [(0, 200), (0, 50)])
    lens = [130, 0]
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.float32)
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu)
    o, lse = lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), out_dtype=torch.float32)
    assert done() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)


@pytest.mark.parametrize("cu", [[0, 40, 20, 60], [-5, 30, 70, 1000], [60, 40, 20, 0], [0, 0, 2 ** 31 - 1, 64]])
def test_paged_fwd_with_offsets_that_do_not_ascend(cu):
    """Offsets are cut to the tokens there are; every row written is a row of q,
    and the rows that one sequence alone names are its rows."""
    q, kp, vp, table, lens, _ = prompt_case(4, 2, 64, 16, [(50, 64), (50, 64), (50, 64)])
    t = q.shape[2] - 128
    big = torch.full((1, 4, t + 16, 64), 7.0, device=DEV)
    lse = torch.full((1, 4, t + 16), 7.0, device=DEV)
    lsx.paged_fwd(q[:, :, :t], kp, vp, table, ints(lens), ints(cu), out=big[:, :, 8:-8], lse=lse[:, :, 8:-8])
    assert done() == 0
    assert big[:, :, :8].eq(7).all() and big[:, :, -8:].eq(7).all()
    assert lse[:, :, :8].eq(7).all() and lse[:, :, -8:].eq(7).all()
    cut = [min(max(c, 0), t) for c in cu]
    named = np.zeros(t, int)
    for a, b in zip(cut, cut[1:]):
        named[a:b] += 1
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.float32)
    for i, (a, b) in enumerate(zip(cut, cut[1:])):
        if b > a:
            only = np.zeros(t, bool)
            only[a:b] = named[a:b] == 1
            fake = [0] * (i + 1) + [b - a] * (3 - i)
            o_ref, l_ref = P.fwd(q[:, :, a:b], kp, vp, table, [n if j == i else 0 for j, n in enumerate(lens)], fake)
            check_close(f64(big[:, :, 8:-8])[:, :, only], o_ref[:, :, only[a:b]], tol)
            check_lse(f64(lse[:, :, 8:-8])[:, :, only], l_ref[:, :, only[a:b]], tol_lse)
    rest = torch.from_numpy(named == 0).to(DEV)
    assert big[:, :, 8:-8][:, :, rest].eq(7).all() and lse[:, :, 8:-8][:, :, rest].eq(7).all()


def test_paged_fwd_equals_decode_on_single_tokens():
    """One new token a sequence: the two entry points agree to P's rounding."""
    lens = [1, 40, 300, 1111]
    q, kp, vp, table, _ = decode_case(8, 2, 1, 128, 32, lens, 0)
    o1, l1 = lsx.paged_decode(q, kp, vp, table, ints(lens), out_dtype=torch.float32)
    packed = q[:, :, 0].transpose(0, 1)[None]
    o2, l2 = lsx.paged_fwd(packed, kp, vp, table, ints(lens), ints([0, 1, 2, 3, 4]), out_dtype=torch.float32)
    assert done() == 0
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16 + P_SPLIT, torch.float32)
    check_close(f64(o2[0].transpose(0, 1)), f64(o1[:, :, 0]), 2 * tol)
    check_lse(f64(l2[0].t()), f64(l1[:, :, 0]), 2 * tol_lse)


# ----------------------------------------------------------- together, streams
def test_serving_steps_together():
    """Prompts of several requests, then decode steps, through page_map,
    page_append, paged_fwd and paged_decode; every answer against the oracle on
    the tokens seen so far."""
    r = np.random.default_rng(5)
    hq, hkv, d, page, b = 8, 2, 128, 16, 5
    n_pages, width = 60, 12
    kp, vp = (torch.full((n_pages, page, hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV).transpose(1, 2)
              for _ in range(2))
    free = [int(x) for x in r.permutation(n_pages)]
    table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
    ctx, hist = [0] * b, [[] for _ in range(b)]
    steps = [[37, 1, 0, 64, 16], [20, 5, 9, 0, 1]] + [[1] * b] * 3 + [[1, 0, 1, 1, 0]]
    for step, new in enumerate(steps):
        total = sum(new)
        slots, cu, lens, taken = lsx.page_map(table, ints(ctx), ints(new), ints(free), page, total + 4)
        n = int(taken)
        assert n <= len(free)
        free = free[n:]
        q = random_tensor((total + 4, hq, d), 900 + step, device=DEV).transpose(0, 1)[None]
        k = random_tensor((total + 4, hkv, d), 920 + step, device=DEV).transpose(0, 1)[None]
        v = random_tensor((total + 4, hkv, d), 940 + step, device=DEV).transpose(0, 1)[None]
        lsx.page_append(k, v, kp, vp, slots)
        at = cu.tolist()
        for i in range(b):
            hist[i] += [(k[0, :, t], v[0, :, t]) for t in range(at[i], at[i + 1])]
        ctx = lens.tolist()
        assert ctx == [len(h) for h in hist]
        if new == [1] * b:
            qq = q[:, :, :b].transpose(0, 2).transpose(1, 2).reshape(b, hq, 1, d)
            o, lse = lsx.paged_decode(qq, kp, vp, table, lens, out_dtype=torch.float32)
            o, lse = o[:, :, 0].transpose(0, 1), lse[:, :, 0].t()
        else:
            o, lse = lsx.paged_fwd(q, kp, vp, table, lens, cu, out_dtype=torch.float32)
            o, lse = o[0], lse[0]
        assert done() == 0
        from oracle import attention as A
        for i in range(b):
            if not new[i]:
                continue
            K, V = (torch.stack([x[j] for x in hist[i]], 1)[None] for j in (0, 1))
            rows = slice(at[i], at[i + 1])
            o_ref, l_ref = A.attn_fwd(f64(q[:, :, rows]), f64(K), f64(V), len(hist[i]) - new[i], 0, True)
            tol, tol_lse = P.tolerances(q, K, V, P_BF16, torch.float32)
            check_close(f64(o[:, rows]), o_ref[0], tol)
            check_lse(f64(lse[:, rows]), l_ref[0], tol_lse)


def test_prefix_equals_the_prefix_in_every_table():
    """A shared prefix of whole pages: the same keys through each sequence's own table."""
    page, prefix_len, lens = 32, 320, [50, 0, 7, 200]
    q, kp, vp, table, prefix = decode_case(8, 2, 1, 128, page, lens, prefix_len)
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), prefix_table=ints(prefix), prefix_len=prefix_len,
                              out_dtype=torch.float32)
    whole = torch.cat([ints(prefix).expand(4, -1), table], 1)
    o2, lse2 = lsx.paged_decode(q, kp, vp, whole, ints([prefix_len + n for n in lens]), out_dtype=torch.float32)
    assert done() == 0
    tol, tol_lse = P.tolerances(q, kp, vp, P_SPLIT, torch.float32)
    check_close(f64(o), f64(o2), 2 * tol)
    check_lse(f64(lse), f64(lse2), 2 * tol_lse)


def test_graph_replays_follow_the_lengths():
    """A captured step replayed with other lengths, tables and rows; two graphs
    with workspaces of their own, replayed in turn on two streams."""
    hq, hkv, d, page, b = 4, 2, 64, 16, 3
    q, kp, vp, table, _ = decode_case(hq, hkv, 1, d, page, [200] * b, 0)
    lens = [ints([200] * b), ints([200] * b)]
    qs = [q.clone(), random_tensor(q.shape, 71, device=DEV)]
    cu = ints([0, 60, 60, 64])
    packed = random_tensor((64, hq, d), 72, device=DEV).transpose(0, 1)[None]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for i in range(2):
        lsx.paged_decode(qs[i], kp, vp, table, lens[i])  # first calls outside the capture
        lsx.paged_fwd(packed, kp, vp, table, lens[i], cu)
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(lsx.paged_decode(qs[i], kp, vp, table, lens[i]) + lsx.paged_fwd(packed, kp, vp, table, lens[i], cu))
        graphs.append(g)
    for new in ([200, 13, 70], [100, 0, 161], [60, 5, 64]):
        for i in range(2):
            lens[i].copy_(ints(new if i == 0 else new[::-1]))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        assert done() == 0
        for i in range(2):
            want = lsx.paged_decode(qs[i], kp, vp, table, lens[i]) + lsx.paged_fwd(packed, kp, vp, table, lens[i], cu)
            assert done() == 0
            for x, y in zip(outs[i], want):
                assert torch.equal(x, y)


def test_calls_on_another_stream_wait_for_nothing_else():
    q, kp, vp, table, _ = decode_case(4, 2, 1, 128, 16, [500, 3], 0)
    lens = ints([500, 3])
    want = lsx.paged_decode(q, kp, vp, table, lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = lsx.paged_decode(q, kp, vp, table, lens)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_views_of_a_fused_projection():
    """q, k and v as slices of one projection row: strides wider than the heads,
    results in q's order of dimensions, the same bits as from dense copies."""
    hq, hkv, d, page, new = 6, 2, 64, 16, [40, 3, 70]
    qkv = random_tensor((sum(new), (hq + 2 * hkv) * d), 8, device=DEV)
    q = qkv[:, :hq * d].view(-1, hq, d).transpose(0, 1)[None]
    k = qkv[:, hq * d:(hq + hkv) * d].view(-1, hkv, d).transpose(0, 1)[None]
    v = qkv[:, (hq + hkv) * d:].view(-1, hkv, d).transpose(0, 1)[None]
    kp, vp = pool(12, hkv, page, d, 1), pool(12, hkv, page, d, 2, token_major=False)
    table = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    slots, cu, lens, _ = lsx.page_map(table, ints([0, 0, 0]), ints(new), ints(list(range(12))), page, sum(new))
    lsx.page_append(k, v, kp, vp, slots)
    kd, vd = kp.clone(), vp.clone()
    lsx.page_append(k.contiguous(), v.contiguous(), kd, vd, slots)
    o, lse = lsx.paged_fwd(q, kp, vp, table, lens, cu)
    o2, lse2 = lsx.paged_fwd(q.contiguous(), kp, vp, table, lens, cu)
    last = [int(x) - 1 for x in cu[1:]]
    q1 = q[0, :, last].transpose(0, 1)[:, :, None]   # [3, Hq, 1, D], one token a sequence
    wide = torch.stack([qkv[i] for i in last])[:, :hq * d].view(3, hq, 1, d)
    o3, lse3 = lsx.paged_decode(wide, kp, vp, table, lens)
    o4, lse4 = lsx.paged_decode(q1.contiguous(), kp, vp, table, lens)
    assert done() == 0
    assert torch.equal(kp, kd) and torch.equal(vp, vd)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(o3, o4) and torch.equal(lse3, lse4)
    assert o[0].transpose(0, 1).is_contiguous()


def test_first_call_of_a_variant_inside_a_capture():
    """Captured without a call before it (heads of 64, 64 rows a key head; 100 heads a key head)."""
    q, kp, vp, table, _ = decode_case(64, 1, 1, 64, 32, [300, 9], 0, seed=77, width=2000)
    lens = ints([300, 9])
    qq, kq, vq, tq, lq, cq = prompt_case(100, 1, 64, 32, [(5, 7), (0, 30)], seed=78)
    args = (qq, kq, vq, tq, ints(lq), ints(cq))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = lsx.paged_decode(q, kp, vp, table, lens) + lsx.paged_fwd(*args)
    g.replay()
    want = lsx.paged_decode(q, kp, vp, table, lens) + lsx.paged_fwd(*args)
    assert done() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_python_refusals():
    q, kp, vp, table, _ = decode_case(4, 2, 1, 128, 16, [50, 3], 0)
    lens = ints([50, 3])
    with pytest.raises(ValueError):
        lsx.paged_decode(q.cpu(), kp, vp, table, lens)
    with pytest.raises(ValueError):
        lsx.paged_decode(q, kp, vp, table, ints([50]))
    with pytest.raises(ValueError):
        lsx.paged_decode(q, kp, vp, table[:1], lens)
    with pytest.raises(TypeError):
        lsx.paged_decode(q, kp, vp, table.long(), lens)
    with pytest.raises(ValueError):
        lsx.paged_decode(q, kp, vp, table, lens, prefix_table=ints([0]), prefix_len=17)
    with pytest.raises(ValueError):
        lsx.paged_fwd(q[:1], kp, vp, table, lens, ints([0, 1]))
    with pytest.raises(lsx._lib.LsxError):
        lsx.paged_decode(q, kp, vp, table, lens, out_dtype=torch.bfloat16, workspace=torch.empty(
            1, dtype=torch.uint8, device=DEV) if lsx.paged_decode_workspace_size(q, kp, 4) > 1 else kp.new_empty(0),
            out=torch.empty((2, 4, 1, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        lsx.page_map(table, ints([0, 0]), ints([1, 1]), ints([5]), 16, -1)
    assert done() == 0
