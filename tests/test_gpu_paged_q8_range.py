"""Rows of an 8-bit cache whose sizes differ widely within a tile of 128 keys: every way
of computing the attention keeps the small ones as far as include/lsx.h says."""

import numpy as np
import pytest
import torch

import long_sequence_exact_gb300 as lsx
import paged_ref as P
import q8_ref as Q
from helpers import f64
from test_gpu_paged import done, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
G, PAGE = 4, 16
FORMS = ["decode", "prefix", "few", "many"]
# roundings of P (bf16 results, f32 ones)
P_BITS = {"decode": (2.0 ** -11, 2.0 ** -22), "prefix": (2.0 ** -11, 2.0 ** -22),
          "few": (2.0 ** -11, 2.0 ** -22), "many": (2.0 ** -8, 2.0 ** -16)}
# an element of K or V of a widened tile is off by this share of the largest one in its
# tile (f16 ends at 2^-24; a row's largest element is above 2^7.8 of its unit and stands at
# 2^7 times that: half of 2^-24 is 2^-39.8 of it); a copy in bf16 loses nothing
FLOOR = {"decode": 0.0, "prefix": 2.0 ** -39, "few": 2.0 ** -39, "many": 0.0}


def cache(k, v, held=True):
    """Rows k, v [n, D] in pages, scattered: (parts, table [1, pages], the rows as held)."""
    k, v = (x.astype(np.float32).astype(np.float64) for x in (k, v))
    n, d = k.shape
    n_pages = -(-n // PAGE)
    order = np.random.default_rng(n).permutation(n_pages + 2)[:n_pages]
    (kp, ks), (vp, vs) = (Q.cache(n_pages + 2, 1, PAGE, d, True, DEV) for _ in range(2))
    slots = [int(order[i // PAGE]) * PAGE + i % PAGE for i in range(n)]
    rows = [torch.from_numpy(x).to(DEV, F32)[None, None] for x in (k, v)]
    lsx.page_append_q8(*rows, kp, ks, vp, vs, ints(slots, torch.int64))
    return (kp, ks, vp, vs), ints(order[None].copy()), [Q.values(*Q.codes(x)) if held else None for x in (k, v)]


def call(form, parts, table, n, q, scale, out_dtype):
    """The query q [D], the same in every row: (o [rows, D], lse [rows], last visible keys)."""
    d = len(q)
    q = torch.from_numpy(q).to(DEV, BF16)
    if form == "decode":
        o, lse = lsx.paged_decode_q8(q.expand(1, G, 1, d).contiguous(), *parts, table, ints([n]), scale,
                                     out_dtype=out_dtype)
        last = np.full((G, 1), n - 1)
    elif form == "prefix":  # 17 sequences without keys of their own, 68 rows
        none = torch.full((17, 1), -1, dtype=torch.int32, device=DEV)
        o, lse = lsx.paged_decode_q8(q.expand(17, G, 1, d).contiguous(), *parts, none, ints([0] * 17), scale,
                                     table[0], n, out_dtype=out_dtype)
        last = np.full((17, G, 1), n - 1)
    else:
        new = 3 if form == "few" else 8 * d // G + 1
        o, lse = lsx.paged_fwd_q8(q.expand(1, G, new, d).contiguous(), *parts, table, ints([n]), ints([0, new]),
                                  scale, out_dtype=out_dtype)
        last = np.broadcast_to(n - new + np.arange(new), (G, new))
    return f64(o).reshape(-1, d), f64(lse).reshape(-1), last.reshape(-1)


def exact(k, v, q, scale, last, ok=None):
    """(o, lse, sums of p |v|, p) of each row, in 64 bits."""
    s = np.where(np.arange(len(k)) <= last[:, None], scale * (k @ q), -np.inf)
    if ok is not None:
        s = np.where(ok, s, -np.inf)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(-1, keepdims=True)
    p = p / total
    return p @ v, (top + np.log(total))[:, 0], p @ np.abs(v), p


def check(form, out_dtype, got, want, score_error, v_floor, arg=32.0):
    """Row by row: a weight is off by its score's error, that of the fp32 argument (half a
    step below `arg`), of the exponential (2^-21), of fp32 sums (2^-19) and of P's rounding."""
    o, lse = got
    o_ref, l_ref, size, _ = want
    rel = score_error + arg * P.U32 + 2.0 ** -21 + 2.0 ** -19
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    assert (np.abs(lse - l_ref) <= rel + np.maximum(np.abs(l_ref), 1.0) * 2 * P.U32).all()
    lim = (2 * rel + P_BITS[form][out_dtype is F32]) * size + v_floor
    if out_dtype is BF16:
        lim = lim + P.U16 * np.abs(o_ref)
    assert (np.abs(o - o_ref) <= lim).all(), np.max(np.abs(o - o_ref) / lim)


# ------------------------------------------------------------------- values
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("weights", ["equal", "one"])
@pytest.mark.parametrize("apart", [15, 24, 25, 28, 31, 40])
@pytest.mark.parametrize("form", FORMS)
def test_small_values_beside_a_large_one(form, apart, weights, d, out_dtype):
    """In every tile a row of V 2^apart times as large as the others, of no weight (exp(-96)
    of theirs); the others share the weight, or one of them has it."""
    r = np.random.default_rng(apart)
    n = 330
    k, v = np.zeros((n, d)), r.uniform(0.2, 1.0, (n, d)) * 448 * 2.0 ** (4 - apart)
    v[:, 3] = 448 * 2.0 ** (4 - apart)
    large = [5, 127, 150, 301]
    v[large] = 448 * 2.0 ** 4
    k[large, 0] = -96.0
    if weights == "one":
        k[17, 0] = 40.0
    q = np.zeros(d)
    q[0] = 1.0
    parts, table, (kh, vh) = cache(k, v)
    o, lse, last = call(form, parts, table, n, q, 1.0, out_dtype)
    assert done() == 0
    want = exact(kh, vh, q, 1.0, last)
    vmax = np.abs(vh).max()
    # decode's weights are off by up to 2^-35 of the largest value, which is shared by all
    floor = (2.0 ** -35 if form == "decode" else FLOOR[form]) * vmax
    # (the arguments, in log2: 40 / ln 2 below 64, 96 / ln 2 of keys that do not count)
    check(form, out_dtype, (o, lse), want, 0.0, floor, 64.0)
    if apart <= 28 and form != "decode":
        assert np.abs(want[0]).max() > 8 * floor  # (a row that is lost would show)


# --------------------------------------------------------------------- keys
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", [15, 24, 25, 28, 31])
@pytest.mark.parametrize("form", FORMS)
def test_small_keys_beside_a_large_one(form, apart, d, out_dtype):
    """A key of 57344 and no weight, beside keys 2^apart times smaller whose scores are
    some units apart."""
    r = np.random.default_rng(100 + apart)
    n = 330
    small = 448 * 2.0 ** (7 - apart)
    k, v = r.uniform(-1.0, 1.0, (n, d)) * small, r.standard_normal((n, d))
    k[:, 0], k[:, 3] = 0.0, small
    k[[5, 201]] = 0.0
    k[[5, 201], 0] = 57344.0
    q = 64.0 * r.choice([-1.0, 1.0], d)
    q[0] = -64.0
    scale = 2.0 ** round(np.log2(4.0 / (64 * small * np.sqrt(d))))
    parts, table, (kh, vh) = cache(k, v)
    o, lse, last = call(form, parts, table, n, q, scale, out_dtype)
    assert done() == 0
    want = exact(kh, vh, q, scale, last)
    counts = want[3].max(0) > 2.0 ** -60
    assert not counts[[5, 201]].any() and np.median(want[3].max(-1)) < 0.9
    error = 2 * (d + 2) * P.U32 * scale * np.linalg.norm(q) * np.linalg.norm(kh[counts], axis=-1).max()
    lost = FLOOR[form] * 57344.0 * np.abs(q).sum() * scale
    assert lost < 1.0  # (rows that are lost move scores by several units)
    vmax = np.abs(vh).max()
    floor = (2.0 ** -35 if form == "decode" else FLOOR[form]) * vmax
    check(form, out_dtype, (o, lse), want, error + lost, floor)


# ------------------------------------------------------ pages that do not exist
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [-39, -100, -8, 7])
@pytest.mark.parametrize("gone", [range(0, 8), range(1, 24), range(8, 16)], ids=["first", "behind", "second"])
@pytest.mark.parametrize("form", FORMS)
def test_small_values_behind_missing_pages(form, gone, size, d, out_dtype):
    """Values of any size behind 128 keys or more without pages, which are left out: the
    weights keep their bits whatever stands in for the missing tiles."""
    r = np.random.default_rng(200 + size)
    n = 430
    k, v = r.standard_normal((n, d)), r.uniform(0.2, 1.0, (n, d)) * 448 * 2.0 ** size
    v[:, 3] = 448 * 2.0 ** size
    q = r.standard_normal(d)
    q = f64(torch.from_numpy(q).to(BF16))
    scale = 0.125
    parts, table, (kh, vh) = cache(k, v)
    ok = np.ones(n, bool)
    for i, g in enumerate(gone):
        table[0, g] = (-1, 1 << 20)[i % 2]
        ok[g * PAGE:(g + 1) * PAGE] = False
    o, lse, last = call(form, parts, table, n, q, scale, out_dtype)
    assert done() == -10
    want = exact(kh, vh, q, scale, last, ok)
    error = 2 * (d + 2) * P.U32 * scale * np.linalg.norm(q) * np.linalg.norm(kh, axis=-1).max()
    # a weight is off by no more than 2^-32 of the largest value (decode 2^-35), as is V
    check(form, out_dtype, (o, lse), want, error, (2.0 ** -32 + FLOOR[form]) * np.abs(vh).max())


# ------------------------------------------------------------- values of zero
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("order", ["behind", "before", "between"])
@pytest.mark.parametrize("large", [57344.0, 1.0, 448 * 2.0 ** -100])
@pytest.mark.parametrize("form", FORMS + ["whole"])
def test_many_keys_of_value_zero(form, large, order, out_dtype):
    """2^17 keys of value 0 and 2^-28 of the weight of one key of a large value (57344: e4m3
    at the end of the exponents' range): they count in the row sums, 2^-11 of them, whatever
    the exponents of their values are.  "whole": a prefix under so many rows that it is not
    cut into pieces, with sums of their own."""
    n, d = (1 << 17) + 384, 64
    k, v = np.zeros((n, d)), np.zeros((n, d))
    k[:, 0] = -28.0
    at = {"behind": 5, "before": n - 200, "between": n // 2 + 7}[order]
    k[at, 0] = 0.0
    v[at] = large
    v[at, 1::2] = -large
    q = np.zeros(d)
    q[0] = 1.0
    scale = float(np.float32(np.log(2)))
    parts, table, _ = cache(k, v, False)
    if form == "whole":
        b = 2 * 152 * 256 // G
        o, lse = lsx.paged_decode_q8(torch.from_numpy(q).to(DEV, BF16).expand(b, G, 1, d).contiguous(), *parts,
                                     torch.full((b, 1), -1, dtype=torch.int32, device=DEV),
                                     torch.zeros(b, dtype=torch.int32, device=DEV), scale, table[0], n,
                                     out_dtype=out_dtype)
        assert bool((o == o[:1, :1]).all()) and bool((lse == lse[0, 0]).all())
        o, lse, last = f64(o[0, :1, 0]), f64(lse[0, :1, 0]), np.array([n - 1])
    else:
        o, lse, last = call(form, parts, table, n, q, scale, out_dtype)
    assert done() == 0
    # (a row's result is that of the key at `at` times its weight)
    seen = last + 1
    total = 1.0 + (seen - 1) * np.exp(-28.0 * scale)
    want = Q.values(*Q.codes(v[at:at + 1])) / total[:, None]
    # arguments in log2 below 2^5, the exponential, sums; P's own rounding is none (2^0)
    rel = 32 * P.U32 + 2.0 ** -21 + 2.0 ** -19
    assert (np.abs(lse - np.log(total)) <= rel + 2 * P.U32).all()
    lim = rel + 2.0 ** -21 + (P.U16 if out_dtype is BF16 else 0.0)
    assert (np.abs(o - want) <= lim * np.abs(want)).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_first_keys_of_value_zero(form, d):
    """Values of 0 in the first tiles, as of padding, and of ordinary size behind: LSE and
    results are as near as with ordinary values throughout."""
    r = np.random.default_rng(300 + d)
    n = 700
    k, v = r.standard_normal((n, d)), r.standard_normal((n, d))
    v[:260] = 0.0
    v[420:560] = 0.0
    q = f64(torch.from_numpy(r.standard_normal(d)).to(BF16))
    scale = 0.125
    parts, table, (kh, vh) = cache(k, v)
    error = 2 * (d + 2) * P.U32 * scale * np.linalg.norm(q) * np.linalg.norm(kh, axis=-1).max()
    for out_dtype in (BF16, F32):
        o, lse, last = call(form, parts, table, n, q, scale, out_dtype)
        assert done() == 0
        want = exact(kh, vh, q, scale, last)
        check(form, out_dtype, (o, lse), want, error, (2.0 ** -32 + FLOOR[form]) * np.abs(vh).max())
