"""Attention over the 4-bit cache on the GPU: scores of every magnitude that FP32 holds, slots
that were never written."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say
from tests.plain64 import U, rounding
from tests.test_attention_gpu import Case
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


def never_written(c, token, params):
    """All bits of a token's codes set, and FP16 patterns `params` as its a and b."""
    import torch

    page, t = divmod(token, c.page)
    part = c.pages[int(c.table[0, page])].view(c.heads, -1)
    g, size = c.d // 32, c.page * c.d // 2
    a, b = (torch.tensor([v & 255, v >> 8], dtype=torch.uint8, device="cuda") for v in params)
    part[:, :size].view(c.heads, c.page, -1)[:, t] = 255
    part[:, size:size + c.page * g * 4].view(c.heads, c.page, g, 2, 2)[:, t] = torch.stack([a, b])
    base = size + c.page * g * 4
    part[:, base:base + size].view(c.heads, c.page // 4, c.d // 2, 4)[:, t // 4, :, P.V_BYTE[t % 4]] = 255
    vp = part[:, base + size:].view(c.heads, c.page // 4, g, 2, 4, 2)
    vp[:, t // 4, :, 0, t % 4], vp[:, t // 4, :, 1, t % 4] = a, b


@pytest.mark.parametrize("params", [(0xFFFF, 0xFFFF), (0x7C00, 0xFC00), (0x7BFF, 0x7BFF), (0x7BFF, 0x0000), (0xFBFF, 0xFBFF),
                                    (0x0000, 0x7C00), (0x7E00, 0x0000)])
@pytest.mark.parametrize("hq,heads,d,nq", [(1, 1, 64, 4), (4, 2, 128, 8), (6, 1, 256, 3), (2, 1, 64, 16), (4, 2, 256, 12), (1, 1, 128, 33),
                                           (8, 2, 64, 12), (4, 1, 128, 16), (4, 1, 64, 60), (2, 2, 128, 130), (3, 1, 256, 70)])
def test_rows_do_not_depend_on_slots_that_only_later_ones_see(hq, heads, d, nq, params):
    """A padded chunk: the last tokens' keys and values were not written, and the pages came as
    they were."""
    import torch

    say("attention never written", hq, heads, d, nq, params)
    for n, last in ((nq, 1), (150, 2), (262, 1)):
        c = Case([max(n, nq)], [nq], hq, heads, d, 32, seed=nq)
        want, wlse = c.run()
        for token in range(c.lens[0] - last, c.lens[0]):
            never_written(c, token, params)
        got, lse = c.run()
        assert torch.isfinite(want).all()
        assert torch.equal(got[:nq - last], want[:nq - last]) and torch.equal(lse[:nq - last], wlse[:nq - last])
