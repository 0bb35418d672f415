"""Paged attention where its state begins and ends: short units over a cluster,
a prompt's first key tile, the streams that calls run on, and refusals."""

import numpy as np
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


def steps(q, kp, vp, table, lens, prefix, packed, cu, rows, slots, free):
    """One call of every paged entry point, each form of decode among them; no copy
    from the host, which would wait for the stream."""
    got = list(lsx.page_map(table.clone(), lens, torch.ones_like(lens), free, 16, 5))
    lsx.page_append(rows, rows, kp, vp, slots)
    for width in (table, torch.nn.functional.pad(table, (0, 2500), value=-1)):
        got += lsx.paged_decode(q, kp, vp, width, lens)
    for n in (1, 40):                                  # few query rows behind a prefix, and many
        qq, tt, ll = q.repeat(n, 1, 1, 1), table.repeat(n, 1), lens.repeat(n)
        got += lsx.paged_decode(qq, kp, vp, tt, ll, prefix_table=prefix, prefix_len=100)
    return got + list(lsx.paged_fwd(packed, kp, vp, table, lens, cu))


def test_calls_run_on_the_current_stream_alone():
    """While the default stream is held by a delay (a second or so), calls on another
    stream finish; they would not if any of their launches went to the default
    stream or waited for it.  And calls on the held stream wait behind the delay."""
    q, kp, vp, table, prefix = decode_case(4, 2, 1, 128, 16, [500, 3], 100)
    lens, prefix, cu = ints([500, 3]), ints(prefix), ints([0, 60, 63])
    packed = random_tensor((63, 4, 128), 7, device=DEV).transpose(0, 1)[None]
    rows, slots = random_tensor((1, 2, 3, 128), 8, device=DEV), ints([3, -1, 17], torch.int64)
    args = (q, kp, vp, table, lens, prefix, packed, cu, rows, slots, ints(list(range(9))))
    want = steps(*args)                                # (and everything loaded and allocated once)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        steps(*args)
    assert done() == 0
    delay = 2_000_000_000                              # clock cycles
    other = torch.zeros(8, device=DEV)
    torch.cuda.synchronize()
    held = torch.cuda.Event()
    torch.cuda._sleep(delay)
    other.fill_(1.0)
    held.record()
    with torch.cuda.stream(side):
        got = steps(*args)
    side.synchronize()
    assert not held.query(), "the calls did not run beside the held stream"
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    ready = torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(delay)
        steps(*args)
        ready.record()
    torch.cuda.default_stream().synchronize()
    assert not ready.query(), "a call on the held stream did not wait"
    assert done() == 0


SHAPE, WORKSPACE, ALIGN, UNSUPPORTED = -2, -6, -4, -5


@pytest.mark.parametrize("prefix_len", [0, 100])
def test_refusals_of_outputs_and_workspaces(prefix_len):
    """Each wrong thing by itself, by its code; the right call beside it runs."""
    q, kp, vp, table, prefix = decode_case(4, 2, 1, 128, 16, [50, 3], prefix_len, width=2500)
    pre = dict(prefix_table=ints(prefix), prefix_len=prefix_len) if prefix_len else {}
    call = lambda **kw: lsx.paged_decode(q, kp, vp, table, ints([50, 3]), **pre, **kw)  # noqa: E731
    need = lsx.paged_decode_workspace_size(q, kp, 2500, prefix_len)
    assert need > 256
    room = torch.empty(need + 512, dtype=torch.uint8, device=DEV)
    room = room[(-room.data_ptr()) % 256:]
    out = lambda d, t=torch.bfloat16: torch.empty((2, 4, 1, d), dtype=t, device=DEV)  # noqa: E731
    for code, kw in ((SHAPE, dict(out=out(64))), (WORKSPACE, dict(workspace=room[:need - 1])),
                     (WORKSPACE, dict(workspace=room[:1])), (ALIGN, dict(workspace=room[16:16 + need])),
                     (SHAPE, dict(lse=torch.empty((2, 4, 2), device=DEV))),
                     (ALIGN, dict(out=torch.empty(2 * 4 * 128 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(2, 4, 1, 128)))):
        with pytest.raises(lsx._lib.LsxError) as e:
            call(**kw)
        assert e.value.code == code, kw.keys()
    want = call()
    got = call(out=out(128), workspace=room[:need])
    assert done() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_of_prompt_outputs_and_workspaces():
    q, kp, vp, table, lens, cu = prompt_case(4, 2, 64, 16, [(600, 40), (0, 9)])
    call = lambda **kw: lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), **kw)  # noqa: E731
    need = lsx.paged_fwd_workspace_size(q, kp, 2, table.shape[1])
    room = torch.empty(need + 512, dtype=torch.uint8, device=DEV)
    room = room[(-room.data_ptr()) % 256:]
    for code, kw in ((SHAPE, dict(out=torch.empty((1, 4, 49, 128), dtype=torch.bfloat16, device=DEV))),
                     (WORKSPACE, dict(workspace=room[:need - 1])), (ALIGN, dict(workspace=room[16:16 + need])),
                     (SHAPE, dict(lse=torch.empty((1, 4, 48), device=DEV)))):
        with pytest.raises(lsx._lib.LsxError) as e:
            call(**kw)
        assert e.value.code == code, kw.keys()
    want = call()
    got = call(workspace=room[:need])
    assert done() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------- calls at the ends of the ranges
def test_prompt_lengths_outside_the_table():
    """A length beyond the table stands for the keys that the table holds, seen from
    tokens that are the last of the length as given."""
    q, kp, vp, table, _, cu = prompt_case(4, 2, 64, 16, [(4, 60), (0, 64), (24, 40)], seed=51)
    tol, tol_lse = P.tolerances(q, kp, vp, P_BF16, torch.float32)
    # 64 keys fit a row of the table
    for lens, status in (([64, -3, 20], 0), ([65, 100, 5000], -10), ([2 ** 31 - 1, -2 ** 31, 64], -10)):
        o_ref, l_ref = P.fwd(q, kp, vp, table, [max(0, n) for n in lens], cu)
        o, lse = lsx.paged_fwd(q, kp, vp, table, ints(lens), ints(cu), out_dtype=torch.float32)
        assert done() == status
        check_lse(f64(lse), l_ref, tol_lse)
        check_close(f64(o), o_ref, tol)


@pytest.mark.parametrize("prefix_len", [0, 50])
@pytest.mark.parametrize("batch", [1000, 20011])
def test_decode_of_a_large_batch(batch, prefix_len):
    lens = [(7 * i) % 41 for i in range(batch)]
    few = 40                                            # tables over the pages of a few sequences
    q, kp, vp, table, prefix = decode_case(4, 2, 1, 64, 16, lens[:few], prefix_len, seed=52)
    pick = torch.tensor([max((j for j in range(few) if lens[j] >= n), key=lambda j: -lens[j]) for n in lens], device=DEV)
    table = table[pick]
    q = random_tensor((batch, 4, 1, 64), 53, device=DEV)
    tol, tol_lse = P.tolerances(q, kp, vp, P_SPLIT, torch.float32)
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), prefix_table=ints(prefix) if prefix_len else None,
                              prefix_len=prefix_len, out_dtype=torch.float32)
    assert done() == 0
    some = list(range(0, batch, 37)) + [batch - 1]
    o_ref, l_ref = P.decode(q[some], kp, vp, table[some], [lens[i] for i in some], prefix, prefix_len)
    check_lse(f64(lse[some]), l_ref, tol_lse)
    check_close(f64(o[some]), o_ref, tol)
    # and every row the same as in a batch of another size
    half = batch // 2
    o2, lse2 = lsx.paged_decode(q[half:], kp, vp, table[half:], ints(lens[half:]),
                                prefix_table=ints(prefix) if prefix_len else None, prefix_len=prefix_len,
                                out_dtype=torch.float32)
    assert done() == 0
    check_close(f64(o[half:]), f64(o2), 2 * tol)
    check_lse(f64(lse[half:]), f64(lse2), 2 * tol_lse)


@pytest.mark.parametrize("token_major", [True, False])
def test_keys_and_values_interleaved_in_one_pool(token_major):
    """Views of one tensor that holds both: pages, heads and rows further apart than
    their sizes; the same bits as from pools of their own."""
    n, page, hkv, d = 40, 32, 3, 128
    shape = (n, 2, page, hkv, d) if token_major else (n, 2, hkv, page, d)
    both = random_tensor(shape, 54, device=DEV)
    kp, vp = (both[:, i].transpose(1, 2) if token_major else both[:, i] for i in (0, 1))
    table, lens = ints([[3, 1, 30, 39, 2, 5], [7, 9, 0, 4, 6, 8]]), ints([190, 33])
    q, cu = random_tensor((2, 6, 1, d), 55, device=DEV), ints([0, 100, 130])
    packed = random_tensor((130, 6, d), 56, device=DEV).transpose(0, 1)[None]
    rows, slots = random_tensor((1, hkv, 2, d), 57, device=DEV), ints([35, 20 * page - 1], torch.int64)
    results = []
    for k, v in ((kp, vp), (kp.contiguous(), vp.contiguous())):
        got = list(lsx.paged_decode(q, k, v, table, lens)) + list(lsx.paged_fwd(packed, k, v, table, lens, cu))
        got += lsx.paged_decode(q, k, v, table, lens, prefix_table=ints([11, 12]), prefix_len=50)
        got += lsx.paged_decode(q.repeat(9, 1, 1, 1), k, v, table.repeat(9, 1), lens.repeat(9),
                                prefix_table=ints([11, 12]), prefix_len=50)
        lsx.page_append(rows, 2 * rows, k, v, slots)
        results.append(got + [k, v])
    assert done() == 0
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_the_longest_sequence(d):
    """2^31 - 512 keys, the most that a table may hold, nearly all of them in one
    page that the table names again and again.  A key with a score of 60 near either
    end outweighs them all (e^60 against 2^31 e^4): a row that sees it is its value,
    one that does not is the mean of the one page."""
    page, pages = 256, 2 ** 23 - 2
    keys = pages * page
    kp, vp = (random_tensor((4, 1, page, d), s, 0.1, device=DEV) for s in (58, 59))
    a = (60 / d ** 0.5) ** 0.5                          # a^2 d / sqrt(d) = 60
    q = torch.full((1, 2, 2, d), a, device=DEV).bfloat16()
    kp[1, 0, page - 1] = q[0, 0, 0]
    kp[2, 0, 5] = q[0, 0, 0]
    table = torch.zeros((1, pages), dtype=torch.int32, device=DEV)
    spike = float(q[0, 0, 0].double().square().sum()) * d ** -0.5
    scores = f64(kp[0, 0]) @ f64(q[0, 0, 0]) * d ** -0.5
    w = np.exp(scores)
    mean, mass = (w @ f64(vp[0, 0])) / w.sum(), np.log(w.sum())
    vmax = float(vp.float().abs().max())
    for at, last in ((None, None), ((pages - 1, 1), page - 1), ((0, 2), 5)):
        table.zero_()
        if at:
            table[0, at[0]] = at[1]
        ws = torch.empty(max(lsx.paged_decode_workspace_size(q, kp, pages), 1), dtype=torch.uint8, device=DEV)
        calls = [lsx.paged_decode(q, kp, vp, table, ints([keys]), workspace=ws, out_dtype=torch.float32),
                 lsx.paged_fwd(q, kp, vp, table, ints([keys]), ints([0, 2]), out_dtype=torch.float32)]
        assert done() == 0
        for o, lse in calls:
            o, lse = f64(o), f64(lse)
            for n in range(2):
                if at and (n == 1 or last != page - 1):     # the last key is the second token's alone
                    ref, ref_l = f64(vp[at[1], 0, last]), spike
                    tol = 2.0 ** -8 * vmax
                else:
                    # sums of up to 2^18 equal terms in fp32 drift by up to 2^-24 of the sum a term
                    ref, ref_l = mean, mass + np.log(pages)
                    tol = 2.0 ** -6 * vmax
                assert np.abs(o[0, :, n] - ref).max() <= tol, (at, n)
                assert np.abs(lse[0, :, n] - ref_l).max() <= 2.0 ** -6, (at, n)
