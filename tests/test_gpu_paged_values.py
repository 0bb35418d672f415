"""Paged attention over the values that its documentation allows: scores whose
level moves along the keys, large and small V."""

import numpy as np
import pytest
import torch

import long_sequence_exact_gb300 as lsx
import paged_ref as P
from helpers import check_close, check_lse, f64
from test_gpu_paged import P_BF16, P_SPLIT, decode_case, done, ints, poison, prompt_case

pytestmark = pytest.mark.gpu

# every way through the two entry points: a call, its queries' weights' rounding
PATHS = ["prompt", "chunk", "prefix_many", "prefix_few", "runs", "clusters"]


class Path:
    """A problem whose keys follow one another in `order`: (pages, page, row) of
    the longest sequence's keys 0, 1, .. (behind the shared prefix, where there is one)."""

    def __init__(self, name, d, keys, seed, new=None):
        page, self.name = 16, name
        if name in ("prompt", "chunk"):
            new = (new or keys) if name == "prompt" else 5
            c = prompt_case(4, 2, d, page, [(keys - new, new), (0, 30)], seed=seed)
            self.q, self.kp, self.vp, self.table, self.lens, self.cu = c
            self.prefix, self.prefix_len, self.p = [], 0, P_BF16
            row, n = self.table[0].tolist(), keys
        else:
            b = {"prefix_many": 20, "prefix_few": 3}.get(name, 2)
            self.prefix_len = keys if name.startswith("prefix") else 0
            self.lens = [7, 0, 40] * 7 if self.prefix_len else [keys, 9]
            self.lens = self.lens[:b]
            c = decode_case(4, 2, 2, d, page, self.lens, self.prefix_len, seed, width=2600 if name == "runs" else None)
            self.q, self.kp, self.vp, self.table, self.prefix = c
            self.p = P_SPLIT
            row, n = (self.prefix, keys) if self.prefix_len else (self.table[0].tolist(), keys)
        self.keys = [(row[i // page], i % page) for i in range(n)]

    def levels(self, levels):
        """Scores near levels[i] for key i of self.keys, near 0 for other keys
        (natural logarithm; noise of about 1 stays)."""
        d, big = self.q.shape[-1], max(1.0, max(abs(x) for x in levels))
        a = (big / d ** 0.5) ** 0.5
        self.q.copy_(self.q.float() * 0.05 + a)
        k = self.kp.float() * 0.05
        pages, rows = (torch.tensor(x, device=k.device) for x in zip(*self.keys))
        k[pages, :, rows] += (torch.tensor(levels, device=k.device) / big * a)[:, None, None]
        self.kp.copy_(k)
        return big

    def reference(self, scale=None):
        if self.name in ("prompt", "chunk"):
            return P.fwd(self.q, self.kp, self.vp, self.table, self.lens, self.cu, scale)
        return P.decode(self.q, self.kp, self.vp, self.table, self.lens, self.prefix, self.prefix_len, scale)

    def run(self, dtype=torch.float32, scale=None):
        if self.name in ("prompt", "chunk"):
            return lsx.paged_fwd(self.q, self.kp, self.vp, self.table, ints(self.lens), ints(self.cu), scale,
                                 out_dtype=dtype)
        return lsx.paged_decode(self.q, self.kp, self.vp, self.table, ints(self.lens), scale,
                                prefix_table=ints(self.prefix) if self.prefix_len else None,
                                prefix_len=self.prefix_len, out_dtype=dtype)

    def check(self, level=0.0, dtype=torch.float32, lost=0.0):
        p = P_BF16 if self.name == "prefix_many" and dtype is torch.bfloat16 else self.p
        tol, tol_lse = P.tolerances(self.q, self.kp, self.vp, p, dtype)
        tol += lost
        # the maximum, its sum with the logarithm and the change of base: half a step of the level each
        tol_lse += 3 * P.U32 * level * 1.4427
        o_ref, l_ref = self.reference()
        poison(self.kp, self.vp, self.table, self.lens, 16, self.prefix, self.prefix_len)
        o, lse = self.run(dtype)
        assert done() == 0
        check_lse(f64(lse), l_ref, tol_lse)
        check_close(f64(o), o_ref, tol)


def profile(name, n):
    x = np.linspace(0.0, 1.0, n)
    tile = np.arange(n) // 128
    return {"rise": 80 * x - 40, "fall": 40 - 80 * x, "steps": np.where(tile % 2 == 0, -30.0, 30.0),
            "spike": np.where(tile == 2, 90.0, 0.0), "hole": np.where(tile == 1, -90.0, 0.0),
            "overflow": np.where(tile >= 3, 200.0, -60.0), "climb": 9.0 * tile}[name].tolist()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("levels", ["rise", "fall", "steps", "spike", "hole", "overflow", "climb"])
def test_levels_that_move_along_the_keys(path, d, levels):
    """The reference that weights are formed against has to follow the scores, up
    and down, tile by tile, with what was summed before it."""
    n = 700
    x = Path(path, d, n, 21)
    x.check(x.levels(profile(levels, n)))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("level2", [24, 21, 9, 7, 0, -7, -9, -20, -36])  # base 2
@pytest.mark.parametrize("exponent", [105, -114])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_and_small_values(path, d, level2, exponent, dtype):
    """V of about 2^105, and of about 2^-114 and one sign, over 700 keys, whatever the
    scores' level.  2^8 n |v|, n = 768, is below 2^127.  A product below 2^-126 may
    be lost: 700 of them, over weights whose sum is at least 1/2 a tile."""
    x = Path(path, d, 700, 22)
    if level2:
        x.levels([level2 / 1.4427] * 700)
    x.vp.copy_((x.vp.float() if exponent > 0 else x.vp.float().abs()) * 2.0 ** exponent)
    assert 2.0 ** 8 * 768 * float(x.vp.float().abs().max()) < 2.0 ** 127
    x.check(abs(level2) / 1.4427, dtype, lost=700 * 2.0 ** -126 / (0.5 * 700 / 128))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("level2", [14, 16])  # base 2: below and above what moves the reference
def test_one_heavy_key_of_every_tile_with_large_values(path, d, level2):
    """All of a tile's weight on one key, whose values are the large ones."""
    n = 700
    x = Path(path, d, n, 25)
    levels = [level2 / 1.4427 if i % 128 == 77 else 0.0 for i in range(n)]
    big = x.levels(levels)
    pages, rows = (torch.tensor(t, device=x.vp.device) for t in zip(*x.keys))
    heavy = torch.tensor([105.0 if i % 128 == 77 else 0.0 for i in range(n)], device=x.vp.device)
    v = x.vp.float()
    v[pages, :, rows] *= (2.0 ** heavy)[:, None, None]
    x.vp.copy_(v)
    assert 2.0 ** 8 * 768 * float(x.vp.float().abs().max()) < 2.0 ** 127
    x.check(big)


@pytest.mark.parametrize("batch,hq,hkv,nq", [(2, 8, 2, 1), (8, 4, 1, 1), (9, 8, 2, 1), (40, 2, 2, 1), (3, 8, 2, 5),
                                             (16, 4, 1, 4), (5, 16, 2, 8), (130, 6, 2, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix_len", [16, 100, 1000])
def test_f32_results_behind_a_prefix_keep_16_bits_of_the_weights(batch, hq, hkv, nq, d, prefix_len):
    """8 to 390 query rows a key head.  A small scale keeps the scores' own error
    far below a bf16 rounding of P, so that the bound sees one."""
    lens = [0, 3, 20][:batch] + [0] * (batch - 3)
    q, kp, vp, table, prefix = decode_case(hq, hkv, nq, d, 16, lens, prefix_len, seed=23)
    scale = 0.002
    tol, tol_lse = P.tolerances(q, kp, vp, P_SPLIT, torch.float32, scale)
    assert tol < 2 * 2.0 ** -14 * float(vp.float().abs().max())
    o_ref, l_ref = P.decode(q, kp, vp, table, lens, prefix, prefix_len, scale)
    poison(kp, vp, table, lens, 16, prefix, prefix_len)
    o, lse = lsx.paged_decode(q, kp, vp, table, ints(lens), scale, ints(prefix), prefix_len, out_dtype=torch.float32)
    assert done() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, tol)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("d", [64, 128])
def test_every_page_of_values_counts_in_a_long_row(path, d):
    """Rows over 6000 keys, each held to a bound of its own size.  With weights
    rounded by u independently, the error of a row of O has a root mean square of at
    most u sqrt(sum_j p_j^2 |v_j|^2) <= u max|v| sqrt(sum_j p_j^2); four times that is
    allowed, and what an error of the scores themselves can do.  At this scale the
    weights are nearly equal, and 16 keys' values in the place of others change a row by
    more than twice its bound (shown on the reference, with a page of V swapped): less
    the error that a right result may have, still more than the bound."""
    scale, n = 0.002, 6000
    x = Path(path, d, n, 24, new=150)
    o_ref, l_ref = x.reference(scale)
    squares = np.exp(x.reference(2 * scale)[1] - 2 * l_ref)   # sum_j p_j^2 of each row
    vmax = float(x.vp.float().norm(dim=-1).max())
    rel = P.score_error(x.q, x.kp, scale) + 2.0 ** -19 + 2.0 ** -21 + 2.0 ** -19
    bound = 4 * x.p * vmax * np.sqrt(squares) + 2 * rel * vmax
    long = squares < 1.5 / n                                   # rows that see all of the longest sequence
    assert long.sum() >= 8
    kept = x.vp.clone()
    a, b = x.keys[3008][0], x.keys[16][0]
    x.vp[a] = kept[b]
    planted = np.linalg.norm(x.reference(scale)[0] - o_ref, axis=-1)
    assert (planted[long] > 2 * bound[long]).all()
    x.vp.copy_(kept)
    poison(x.kp, x.vp, x.table, x.lens, 16, x.prefix, x.prefix_len)
    o, lse = x.run(scale=scale)
    assert done() == 0
    fin = np.isfinite(l_ref)
    error = np.linalg.norm(f64(o) - o_ref, axis=-1)
    assert (error[fin] <= bound[fin]).all(), float((error[fin] / bound[fin]).max())
    check_lse(f64(lse), l_ref, rel + 2.0 ** -19)
