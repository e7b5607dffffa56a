"""Sampling on the GPU where a part's largest logit lies on the border of its first bin: rows
of zeros, one-hot and sparse rows, in either order of their parts."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say
from tests.test_kv_gpu import dt
from tests.test_sample_gpu import dev

pytestmark = pytest.mark.gpu

NONE = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def may_be_kept(y, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Tokens that the filters keep, those among them whose decision is closer than 2^-34 of the
    sums (what FP64's sums of up to 2^20 weights may lose, and more than the weights' 2^-40)."""
    y = y.astype(np.float64)
    top_p, min_p, temperature = (float(np.float32(v)) for v in (top_p, min_p, temperature))
    order = np.argsort(-y, kind="stable")
    w = np.exp((y[order] - y.max()) / temperature)
    if 0 < top_k < len(y):
        w[top_k:] = 0.0
    keep = w > 0
    if top_p < 1.0:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep &= before < (top_p + 2.0 ** -34) * w.sum()
    if min_p > 0.0:
        keep &= w >= min(min_p, 1.0) * (1 - 2.0 ** -34)
    keep[0] = True
    out = np.zeros(len(y), bool)
    out[order[keep]] = True
    return out


def check_rows(rows, settings, u, y="f32"):
    """Every row with its settings: the token of the definition where its nearest decision is
    clear, one that may be kept where it is not; the same bits again and again."""
    import torch

    yt = torch.from_numpy(np.stack(rows).astype(np.float32)).to(dt(y)).cuda()
    s = {key: [{**NONE, **row}[key] for row in settings] for key in NONE}
    args = (dev(u), dev(s["temperature"]), dev(s["top_k"], "int32"), dev(s["top_p"]), dev(s["min_p"]))
    idx, prob = lowbit.lowbit_sample(yt, *args)
    for _ in range(3):
        again = lowbit.lowbit_sample(yt, *args)
        assert torch.equal(again[0], idx) and torch.equal(again[1], prob)
    values, idx, prob = yt.double().cpu().numpy(), idx.tolist(), prob.double().cpu().numpy()
    clear = 0
    for i, row in enumerate(settings):
        token, p, margin = P.sample(values[i], u[i], **row)
        if margin > 2.0 ** -34:
            clear += 1
            assert idx[i] == token, (i, row, u[i], idx[i], token)
            assert abs(prob[i] - p) <= p * (2.0 ** -23 + 2.0 ** -36), (i, prob[i], p)
        else:
            assert may_be_kept(values[i], **row)[idx[i]], (i, row, u[i], idx[i])
    return idx, clear


ONE_HOT = [  # logits, value and place of the one that is not 0, settings
    (8000, 3.0, 5000, dict(top_k=20)), (151936, 20.0, 151935, dict(top_k=1000)), (8000, 2.0, 7999, dict(top_p=0.9)),
    (8000, 2.0, 7999, dict(top_k=4500, top_p=0.6)), (40000, 4.0, 39999, dict(top_k=9000, top_p=0.5)),
    (40000, 1.0, 20000, dict(top_p=0.3)), (40000, 0.1, 30000, dict(min_p=0.91)), (151936, 5.0, 9, dict(top_k=8192)),
    (151936, 1e-3, 151935, dict(top_p=0.999)), (9000, 2.5, 8999, dict()), (151936, 9.0, 77777, dict(top_k=8193)),
    (30000, 30.0, 29000, dict(top_k=3, top_p=0.999))]


@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("n,peak,at,kw", ONE_HOT)
def test_one_logit_over_zeros(n, peak, at, kw, reverse, y):
    say("sample one-hot", n, peak, at, kw, reverse, y)
    row = np.zeros(n)
    row[at] = peak
    if reverse:
        row = row[::-1].copy()
    u = [0.0, 2.0 ** -24, 0.03, 0.3, 0.5, 0.8, 0.97, 1.0 - 2.0 ** -24] * 3
    settings = [dict(kw, temperature=t) for t in (1.0, 0.5, 1.3) for _ in range(8)]
    idx, clear = check_rows([row] * 24, settings, u, y)
    assert clear >= 12
    # u = 0: the first token that is kept, of those that weigh (2^-43 is more than the least of any n here)
    for i in range(0, 24, 8):
        weighs = np.exp((row - row.max()) / settings[i]["temperature"]) > 2.0 ** -43
        assert idx[i] == np.nonzero(may_be_kept(row, **settings[i]) & weighs)[0][0]


@pytest.mark.parametrize("sign", [0.0, -0.0])
def test_parts_of_zeros_and_others(sign):
    """Zeros as the largest of some parts, above and below what other parts have; both zeros alike."""
    say("sample zeros among parts", sign)
    g = np.random.default_rng(31)
    n = 30000
    rows, settings = [], []
    for gap in (0.25, 1.0, 4.0, 11.0, 25.0):
        for kw in (dict(), dict(top_k=50), dict(top_k=4097), dict(top_k=9500), dict(top_p=0.7), dict(min_p=0.2),
                   dict(top_k=6000, top_p=0.8, min_p=1e-3)):
            part = np.arange(n) // 4096
            y = np.where(part % 3 == 0, sign, np.where(part % 3 == 1, -gap, gap / 2))
            y[g.integers(0, n, 200)] = -np.inf
            y[g.integers(0, n, 50)] = sign
            y[g.integers(0, n, 3)] = gap
            rows.append(y)
            settings.append(kw)
    for shift in range(3):  # the parts in other orders
        check_rows([np.roll(r, shift * 4096) for r in rows], settings, g.random(len(rows)))
    check_rows([r[::-1].copy() for r in rows], settings, g.random(len(rows)))


@pytest.mark.parametrize("n,behind", [(2, [-33.9, -34.0, -34.2]), (4096, [-33.9, -34.0, -34.2]), (1 << 14, [-33.2, -33.3]),
                                      (151936, [-30.45, -30.55]), (1 << 20, [-29.1, -29.2])])
def test_the_least_weights_that_count(n, behind):
    """One logit behind another, which is a whole octave: with u = 0 it is drawn if it weighs
    something.  A weight is cut to a whole number of 2^-unit.  In the part of the largest it has been
    rounded to one of 2^-51 before, so it counts from 1 - 2^(unit - 52) of 2^-unit on there, which is
    7/8 at unit 49 (a logit of -34.098); in another part its own base is 48 octaves lower, and that
    rounding no matter."""
    unit = min(49, 62 - int(np.ceil(np.log2(n))))
    for first, last in ((0, n - 1), (n // 2 - 1, n // 2)):
        least = (1 - (2.0 ** (unit - 52) if first // 4096 == last // 4096 else 0.0)) * 2.0 ** -unit
        rows = np.full((len(behind), n), -np.inf)
        rows[:, last] = 0.0
        rows[:, first] = behind
        idx, prob = lowbit.lowbit_sample(dev(rows), dev([0.0] * len(behind)))
        w = np.exp(np.float32(behind).astype(np.float64))
        assert (np.abs(w / least - 1) > 1e-3).all() and w[0] > least > w[-1]
        assert idx.tolist() == [first if v > least else last for v in w]
        assert abs(float(prob[0]) / w[0] - 1) < 1e-5


@pytest.mark.parametrize("sigma", [4.0, 15.0, 60.0])
def test_every_token_is_one_that_the_filters_keep(sigma):
    """Rows so uneven that the nearest decision is often closer than the weights' steps."""
    say("sample uneven", sigma)
    g = np.random.default_rng(int(sigma))
    n = 20000
    rows, settings = [], []
    for i in range(48):
        y = g.standard_normal(n) * sigma
        y[g.integers(0, n, 4000)] = np.float32(y.max() - (i % 8))
        rows.append(y.astype(np.float32))
        settings.append(dict(temperature=float(g.choice([0.3, 1.0, 2.0])), top_k=int(g.choice([0, 3, 700, 4001, 9000])),
                             top_p=float(g.choice([0.2, 0.9, 0.9999, 1.0])), min_p=float(g.choice([0.0, 0.01, 0.5]))))
    check_rows(rows, settings, g.choice([0.0, 1e-7, 0.5, 1.0], 48))
