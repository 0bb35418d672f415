"""Paged attention where its state begins and ends: short units over a cluster,
a prompt's first key tile, the streams that calls run on, and refusals."""

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
