"""Paged attention where its state begins and ends: short units over a cluster,
a prompt's first key tile."""

import pytest
import torch

import long_sequence_exact_gb300 as lsx
import paged_ref as P
from helpers import check_close, check_lse, f64
from long_sequence_exact_gb300.inputs import random_tensor
from test_gpu_paged import DEV, P_BF16, P_SPLIT, decode_case, done, ints, poison, prompt_case

pytestmark = pytest.mark.gpu


def level_scores(q, kp, level, scale):
    """q and kp moved so that every score lies near `level`: q = a + noise,
    k = +-a + noise with D a^2 scale = |level|."""
    a = (abs(level) / (q.shape[-1] * scale)) ** 0.5
    q.copy_(q.float() * 0.05 + a)
    kp.copy_(kp.float() * 0.05 + (a if level > 0 else -a))


@pytest.mark.parametrize("level", [0, -120])
@pytest.mark.parametrize("hq,nq", [(2, 1), (14, 3), (24, 5)])  # 1, 21 and 60 rows a key head
@pytest.mark.parametrize("d", [64, 128])
def test_clusters_with_fewer_steps_than_blocks(d, hq, nq, level):
    """Units of 0 to 9 steps (64 keys of 128, 128 keys of 64) over clusters of
    eight: blocks without a step of their own hold no keys, at whatever level the
    scores of the others are (weights of 2^-173 against a maximum of 0 vanish)."""
    step, page = 8192 // d, 16
    lens = sorted({max(0, i * step + x) for i in range(10) for x in (0, 1)})[:19]
    assert len(lens) == 19 and lens[0] == 0 and lens[-1] == 9 * step
    q, kp, vp, table, _ = decode_case(hq, 2, nq, d, page, lens, 0, seed=31)
    assert lsx.paged_decode_workspace_size(q, kp, table.shape[1]) == 0  # the form without partials
    if level:
        level_scores(q, kp, level, d ** -0.5)
    tol, tol_lse = P.tolerances(q, kp, vp, P_SPLIT, torch.float32)
    # the maximum, its sum with the logarithm and the change of base: half a step of the level each
    tol_lse += 3 * P.U32 * abs(level) * 1.4427
    o_ref, l_ref = P.decode(q, kp, vp, table, lens)
    poison(kp, vp, table, lens, page)
    for _ in range(3):
        random_tensor((1 << 22,), 1, 1e30, device=DEV)  # other values in registers and shared memory
        o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), out_dtype=torch.float32)
        assert done() == 0
        check_lse(f64(lse), l_ref, tol_lse)
        check_close(f64(o), o_ref, tol)


@pytest.mark.parametrize("level", [60, -60])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_the_first_tile_formed_twice(d, level):
    """Rows that end in their first tile, and first tiles whose scores lie far from
    0, form their weights a second time in the same place: a weight left from the
    first time would be 2^86 or 2^-86 times too large.  Thirty times the same bits."""
    seqs = [(0, 100), (0, 1), (20, 60), (0, 0), (0, 700), (130, 40)]
    q, kp, vp, table, lens, cu = prompt_case(4, 2, d, 16, seqs, seed=41)
    level_scores(q, kp, level, d ** -0.5)
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.float32)
    tol_lse += 3 * P.U32 * abs(level) * 1.4427
    o_ref, l_ref = P.fwd(q, kp, vp, table, lens, cu)
    poison(kp, vp, table, lens, 16)
    args = (q, kp, vp, table, ints(lens), ints(cu))
    o, lse = lsx.paged_fwd(*args, out_dtype=torch.float32)
    assert done() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)
    for _ in range(30):
        o2, lse2 = lsx.paged_fwd(*args, out_dtype=torch.float32)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert done() == 0
