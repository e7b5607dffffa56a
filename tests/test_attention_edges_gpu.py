"""Attention over the 4-bit cache on the GPU: scores of every magnitude that FP32 holds."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say
from tests.plain64 import U, rounding
from tests.test_kv_gpu import dt, host, i32

pytestmark = pytest.mark.gpu

SHAPES = [(64, 1, 1), (128, 2, 1), (256, 6, 1), (128, 8, 4), (256, 2, 10), (64, 4, 12), (128, 1, 100), (256, 1, 100)]


@pytest.mark.parametrize("size", [1.0, 1e9, 1e20, 1e29, 1e31, 1e35, 2e37])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("d,group,nq", SHAPES)
def test_rows_whose_scores_are_all_far_from_zero(d, group, nq, sign, size):
    """Keys of 8 or of 16 in front: the larger scores share the row, however large all are."""
    import torch

    say("attention far scores", d, group, nq, sign, size)
    n, page = 300, 16
    g = torch.Generator(device="cuda").manual_seed(d + nq)
    k = torch.zeros(n, 1, d, device="cuda")
    k[:, 0, 0] = 8.0
    k[::3, 0, 0] = 16.0
    v = torch.randn(n, 1, d, generator=g, device="cuda")
    pages = torch.zeros(19, P.page_bytes(1, d, page), dtype=torch.uint8, device="cuda")
    slots = i32(np.arange(n))
    lowbit.lowbit_kv_store(k, v, slots, pages, page)
    kk, vv = (host(t)[:, 0] for t in lowbit.lowbit_kv_load(pages, page, slots, 1, d))
    q = torch.zeros(2 * nq, group, d, device="cuda")
    q[:, :, 0] = sign * size / 8.0
    q = q.to(dt("bf16"))
    for scale in (1.0, -1.0):
        lse = torch.zeros(2 * nq, group, device="cuda")
        out = lowbit.lowbit_attention(q, pages, page, i32([np.arange(19)] * 2), i32([n, n]), q_start=i32([0, nq, 2 * nq]),
                                      max_q=nq, scale=scale, lse=lse, out_dtype=dt("f32"))
        got, glse, qv = host(out), host(lse), float(q[0, 0, 0])
        for row in {0, nq - 1, 2 * nq - 1}:
            last = n - nq + row % nq
            s = kk[:last + 1, 0] * qv * scale
            p = np.exp(s - s.max())
            # equal scores have equal weights; size 1: scores of 1 and 2, each off by some U of itself
            err = 2.0 ** -11 + 2.0 ** -20
            want = p @ vv[:last + 1] / p.sum()
            bound = err * (p @ (np.abs(vv[:last + 1]) + np.abs(want))) / p.sum() * 1.01
            bound = bound + rounding(np.abs(want) + bound, "float32")
            assert (np.abs(got[row] - want) <= bound).all(), (scale, row)
            wlse = s.max() + np.log(p.sum())
            assert (np.abs(glse[row] - wlse) <= abs(wlse) * 8 * U + 2.0 ** -10).all(), (scale, row)
