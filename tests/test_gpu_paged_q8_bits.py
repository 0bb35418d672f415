"""The bits of P that include/lsx.h states for each way of computing attention over an
8-bit cache, and bounds that a lost or doubled rescaling of O does not pass."""

import numpy as np
import pytest
import torch

import long_sequence_exact_gb300 as lsx
import paged_ref as P
from helpers import check_close, check_lse, f64
from test_gpu_paged import PROMPT, check_prompt, done, ints
from test_gpu_paged_q8_attention import P_F16, P_F16X2, decode, decode_case, prompt_case, tolerances

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def by_copy(q, c, batch, width):
    return (lsx.paged_fwd_q8_workspace_size(q, c.kp, batch, width) >
            lsx.paged_fwd_q8_workspace_size(q, c.kp, batch, width, copy=False))


@pytest.mark.parametrize("case", PROMPT + [
    (32, 8, 128, 16, [(2000, 30)]), (8, 8, 64, 32, [(700 + 50 * i, 3 + 20 * i) for i in range(5)]),
    (16, 1, 128, 256, [(0, 100), (513, 40)]), (64, 1, 64, 32, [(300, 9), (0, 8), (90, 10)]),
], ids=lambda c: "-".join(map(str, c[:4])) + f"-{len(c[4])}")
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_fwd(case, out_dtype):
    q, c, table, lens, cu = prompt_case(*case, seed=160, token_major=out_dtype is BF16, tail=3)
    dense = c.dense()
    copied = by_copy(q, c, len(lens), table.shape[1])
    bits = ((2.0 ** -8, 2.0 ** -16) if copied else (P_F16, P_F16X2))[out_dtype is F32]
    tol, tol_lse = P.tolerances(q, *dense, bits, out_dtype)
    # (a weight in place is off by up to half of 2^-24 in units of 2^-8 of the largest value:
    # fewer than 2^13 keys, against a sum of weights of 1 and more)
    tol += 0.0 if copied else 2.0 ** -20 * float(dense[1].float().abs().max())
    o_ref, l_ref = P.fwd(q, *dense, table, lens, cu)
    c.poison(table, lens, case[3])
    out = torch.full(q.shape, 7.0, dtype=out_dtype, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    lsx.paged_fwd_q8(q, *c.parts, table, ints(lens), ints(cu), out=out, lse=lse)
    assert done() == 0
    check_prompt(out, lse, o_ref, l_ref, tol, tol_lse)


@pytest.mark.parametrize("rows", [33, 64, 65, 130])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_prefix_of_many_rows(rows, d, out_dtype):
    lens = [(29 * i) % 40 for i in range(rows)]
    case = (2, 2, 1, d, 32, lens, 1500)
    q, c, table, prefix = decode_case(*case, seed=150, token_major=out_dtype is F32)
    dense = c.dense()
    tol, tol_lse = tolerances(q, dense, P_F16X2 if out_dtype is F32 else P_F16, out_dtype)
    o_ref, l_ref = P.decode(q, *dense, table, lens, prefix, 1500)
    o, lse = decode(q, c, table, lens, prefix, 1500, out_dtype=out_dtype)
    assert done() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)


# ------------------------------------------------------------- values of many sizes
ORDERS = {"rise": lambda x: x, "fall": lambda x: 1 - x, "mixed": lambda x: (x * 701 // 1 * 7 % 31) / 31,
          "last": lambda x: (x > 0.998).astype(float), "first": lambda x: (x < 0.004).astype(float)}


def sized_case(d, keys, order, span, form):
    """One sequence (a prefix under 17 x 4 rows) whose values grow by 2^span in the order
    given, with scores that make up for them: weights 2^-e, values 2^e."""
    n, page, hkv = 700, 16, 2
    b = 17 if form == "prefix" else 1
    new = {"few": 3, "many": 8 * d // 4 + 1}.get(form, 1)
    q, c, table, prefix = decode_case(8, hkv, 1, d, page, [n], 0, seed=170, width=keys // page, spread=0)
    e = np.round(span * ORDERS[order](np.arange(n) / (n - 1.0))).astype(int)
    pos = np.arange(n)
    at = table[0].cpu().numpy()[pos // page] * page + pos % page
    exps = np.zeros(c.kp.shape[0] * page, int)
    exps[at] = e
    exps = torch.from_numpy(exps).to(DEV).view(-1, 1, page)
    c.vs.copy_((105 + exps).expand_as(c.vs))
    kd = torch.zeros(1, hkv, c.kp.shape[0] * page, d, device=DEV)
    kd[..., 0] = -exps.reshape(-1).float()
    lsx.page_append_q8(kd, kd, c.kp, c.ks, c.vp.clone(), c.vs.clone(), torch.arange(kd.shape[2], device=DEV))
    q = torch.zeros((b, 8, new, d) if form in ("decode", "prefix") else (1, 8, new, d), dtype=BF16, device=DEV)
    q[..., 0] = 1.0
    return q, c, table, n, new, b


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("d,keys", [(64, 0), (128, 40000)])
@pytest.mark.parametrize("form", ["decode", "prefix", "few", "many"])
def test_rescaled_values(form, order, d, keys):
    """Each row within what is kept of its weights' sum of p |v|, and of the largest value
    seen; results of 0, of twice the size and of half are not within it."""
    span, scale = 15, float(np.log(2))
    q, c, table, n, new, b = sized_case(d, keys, order, span, form)
    kd, vd = (f64(x) for x in c.dense())
    pages = table[0].cpu().numpy()[: -(-n // 16)]
    kd, vd = (x[pages].transpose(1, 0, 2, 3).reshape(2, -1, d)[:, :n] for x in (kd, vd))
    for dtype in (F32, BF16):
        if form == "decode":
            o, lse = lsx.paged_decode_q8(q, *c.parts, table, ints([n]), scale, out_dtype=dtype)
        elif form == "prefix":
            none = torch.full((b, 1), -1, dtype=torch.int32, device=DEV)
            o, lse = lsx.paged_decode_q8(q, *c.parts, none, ints([0] * b), scale, table[0, : len(pages)], n, out_dtype=dtype)
        else:
            o, lse = lsx.paged_fwd_q8(q, *c.parts, table, ints([n]), ints([0, new]), scale, out_dtype=dtype)
        assert done() == 0
        last = n - 1 if form in ("decode", "prefix") else n - new + np.arange(new)
        o, lse = f64(o), f64(lse)
        bits = ((2.0 ** -8, 2.0 ** -16) if form == "many" else (P_F16, P_F16X2))[dtype is F32]
        floor = {"decode": 2.0 ** -36, "many": 2.0 ** -100}.get(form, 2.0 ** -33)
        for h in range(2):
            s = np.where(np.arange(n) <= np.reshape(last, (-1, 1)), scale * kd[h, :, 0], -np.inf)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            l_ = p.sum(-1, keepdims=True)
            want, size = p @ vd[h] / l_, p @ np.abs(vd[h]) / l_
            # arguments below 2^5 in log2, the exponential, sums; LSEs below 64
            rel = 2.0 ** -19 + 2.0 ** -21 + 2.0 ** -19
            vmax = np.abs(vd[h]).max()
            lim = (2 * rel + bits) * size + floor * n * vmax / l_ + (P.U16 if dtype is BF16 else 0) * np.abs(want)
            got = o[:, 4 * h:4 * h + 4]
            assert (np.abs(lse[:, 4 * h:4 * h + 4] - (top + np.log(l_))[:, 0]) <= rel + 2.0 ** -19).all()
            assert (np.abs(got - want) <= lim).all()
            # the bound sees what it is there for
            for wrong in (0.0, 0.5, 2.0):
                assert (np.abs(wrong * want - want) > lim).any(-1).all()
