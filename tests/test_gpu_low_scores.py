"""Rows whose scores are all far below zero (or far above): the running maximum
has to be that of the scores alone.  A maximum that something else entered, a
zero for instance, underflows every weight of such a row: O = 0, LSE = -inf."""

import pytest
import torch

import long_sequence_exact_gb300 as lsx
from helpers import TOL_O_BF16, check_close, check_lse, f64
from long_sequence_exact_gb300.inputs import random_tensor
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("level", [-400.0, -100.0, 100.0, 400.0])
@pytest.mark.parametrize("n", [300, 512])
def test_forward_with_every_score_near_a_level(d, level, n):
    # q = a + noise, k = +-a + noise with d * a^2 / sqrt(d) = |level|
    a = (abs(level) / d ** 0.5) ** 0.5
    q = (random_tensor((1, 4, n, d), 1, 0.01, dtype=torch.float32, device=DEV) + a).bfloat16()
    k = random_tensor((1, 2, n, d), 2, 0.01, dtype=torch.float32, device=DEV) + (a if level > 0 else -a)
    k = k.bfloat16()
    v = random_tensor((1, 2, n, d), 3, device=DEV)
    # scores are sums of d products of size a^2 in fp32: off by at most
    # 2 (d + 2) half steps (2^-24) of their size, about |level|
    tol_lse = 2 * (d + 2) * 2.0 ** -24 * abs(level) * 1.1 + 1e-5
    for causal in (True, False):
        o_ref, l_ref = A.attn_fwd(f64(q), f64(k), f64(v), 0, 0, causal)
        for o, lse in (lsx.chunked_fwd(q, k, v, 256, causal), lsx.chunk_fwd(q, k, v, 0, 0, causal),
                       lsx.chunk_fwd(q, k, v, 0, 0, causal, use_workspace=False)):
            torch.cuda.synchronize()
            assert lsx.sync_status() == 0
            check_lse(f64(lse), l_ref, tol_lse)
            check_close(f64(o), o_ref, TOL_O_BF16)
    # the same rows from pages, as a prompt and as single tokens
    page = 16
    pages = -(-n // page)
    kp, vp = (torch.zeros(2, pages * page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kp[:, :n], vp[:, :n] = k[0], v[0]
    kp, vp = (x.view(2, pages, page, d).transpose(0, 1) for x in (kp, vp))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o_ref, l_ref = A.attn_fwd(f64(q), f64(k), f64(v), 0, 0, True)
    o, lse = lsx.paged_fwd(q, kp, vp, table, lens, cu)
    o1, lse1 = lsx.paged_decode(q[:, :, -1:], kp, vp, table, lens)
    torch.cuda.synchronize()
    assert lsx.sync_status() == 0
    check_lse(f64(lse), l_ref, tol_lse)
    check_close(f64(o), o_ref, TOL_O_BF16)
    check_lse(f64(lse1), l_ref[:, :, -1:], tol_lse)
    check_close(f64(o1), o_ref[:, :, -1:], TOL_O_BF16)
