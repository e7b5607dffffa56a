"""Sampling on the GPU against the 64-bit form: every filter and their
combinations, ties, few and many kept tokens, rows without a way on."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say
from tests.test_kv_gpu import dt

pytestmark = pytest.mark.gpu


def dev(a, dtype="float32"):
    import torch

    return torch.tensor(np.asarray(a).tolist(), dtype=getattr(torch, dtype), device="cuda")


def check(y, u, temperature=None, top_k=None, top_p=None, min_p=None, least=None, **kw):
    """y: GPU tensor [b][n].  Rows whose nearest decision is further than 2^-34
    of the sums from falling the other way have to give the token; 2^-40 is what the
    weights are off by, and FP64's sums of up to 2^20 of them lose less than 2^-34.
    Returns how many rows were that clear."""
    opt = lambda v, dtype="float32": None if v is None else dev(v, dtype)  # noqa: E731
    idx, prob = lowbit.lowbit_sample(y, dev(u), opt(temperature), opt(top_k, "int32"), opt(top_p), opt(min_p), **kw)
    idx, prob, values = idx.cpu().numpy(), prob.double().cpu().numpy(), y.double().cpu().numpy()
    clear = 0
    for i in range(y.shape[0]):
        at = lambda v, none: none if v is None else v[i]  # noqa: E731
        token, p, margin = P.sample(values[i], u[i], at(temperature, 1.0), at(top_k, 0), at(top_p, 1.0), at(min_p, 0.0))
        if margin > 2.0 ** -34:
            clear += 1
            assert idx[i] == token, (i, idx[i], token, margin)
            assert abs(prob[i] - p) <= p * (2.0 ** -23 + 2.0 ** -36), (i, prob[i], p)
        else:
            assert 0 <= idx[i] < y.shape[1] and 0 < prob[i] <= 1
    assert clear >= (y.shape[0] * 0.9 if least is None else least)
    return idx


def logits(g, b, n, sigma, y="f32"):
    import torch

    return torch.from_numpy((g.standard_normal((b, n)) * sigma).astype(np.float32)).to(dt(y)).cuda()


@pytest.mark.parametrize("y", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 63, 1000, 4095, 4096, 4097, 32003, 151936])
def test_settings_side_by_side(y, n):
    say("sample", y, n)
    g = np.random.default_rng(n)
    b = 24
    yt = logits(g, b, n, 2.0, y)
    t = g.choice([0.2, 0.5, 1.0, 1.7], b)
    k = g.choice([0, 1, 5, 20, 300, 5000, n, n + 9, -3], b)
    p = g.choice([0.1, 0.5, 0.85, 0.99, 1.0, 1.0], b)
    mp = g.choice([0.0, 0.0, 0.001, 0.05, 0.4], b)
    check(yt, g.random(b), t, k, p, mp)


@pytest.mark.parametrize("sigma", [0.0, 0.01, 1.0, 5.0, 50.0])
@pytest.mark.parametrize("which", ["open", "top_k", "top_p", "min_p", "all"])
def test_few_and_many_kept_tokens(sigma, which):
    """From all tokens alike to one that has everything; cuts that leave thousands."""
    say("sample kept", sigma, which)
    g = np.random.default_rng(int(sigma * 100) + len(which))
    b, n = 10, 40000
    y = logits(g, b, n, sigma)
    kw = {}
    if which in ("top_k", "all"):
        kw["top_k"] = [2000, 2047, 2048, 2049, 2500, 5000, 12345, 30000, 39999, 1]
    if which in ("top_p", "all"):
        kw["top_p"] = [0.01, 0.05, 0.1, 0.3, 0.5, 0.7, 0.9, 0.95, 0.999, 1e-6]
    if which in ("min_p", "all"):
        kw["min_p"] = [1e-6, 1e-4, 1e-3, 0.01, 0.03, 0.1, 0.3, 0.5, 0.9, 1.0]
    check(y, g.random(b), **kw)


@pytest.mark.parametrize("levels", [1, 2, 7, 40])
def test_values_that_many_tokens_share(levels):
    """Ties at the cuts go to the lowest numbers, thousands of them too."""
    import torch

    say("sample ties", levels)
    g = np.random.default_rng(levels)
    b, n = 24, 50000
    y = torch.from_numpy(g.integers(0, levels, (b, n)).astype(np.float32) / 4).cuda()
    k = [0, 1, 2, 100, 2048, 2049, 4096, 4097, 10000, 25001, 49999, 7] * 2
    p = [1.0] * 12 + [0.3, 0.999, 0.5, 0.25, 0.75, 0.1, 0.5, 0.9, 0.123, 0.6, 0.7, 0.01]
    check(y, g.random(b), top_k=k, top_p=p, least=0)
    # which of the equal ones stay is known whatever the sums do
    for k1, i in ((3000, 5), (1, 0), (2048, 3), (2049, 4)):
        row = y[i:i + 1]
        order = np.argsort(-row[0].cpu().numpy(), kind="stable")[:k1]
        idx, _ = lowbit.lowbit_sample(row, dev([1.0]), top_k=dev([k1], "int32"))
        assert int(idx) == order.max()  # u next to 1: the last kept number
        idx, _ = lowbit.lowbit_sample(row, dev([0.0]), top_k=dev([k1], "int32"))
        assert int(idx) == order.min()


def test_edges_of_the_random_number_and_settings():
    g = np.random.default_rng(3)
    nan, inf = float("nan"), float("inf")
    y = logits(g, 1, 5000, 1.0).repeat(12, 1)
    u = [0.0, -1.0, nan, 1.0, 5.0, inf, 1 - 2.0 ** -24, 2.0 ** -30, 0.5, 0.5, 0.5, 0.5]
    check(y, u, temperature=[1.0] * 8 + [nan, -1.0, 1e-9, 0.0], least=12)
    check(y, [0.3] * 12, top_p=[nan, 0.0, -1.0, 2.0, inf, 1.0, 1e-30, 0.5, 0.5, 0.5, 0.5, 0.5],
          min_p=[0, 0, 0, 0, 0, 0, 0, nan, -2.0, 1.0, 3.0, 1e-30], least=12)
    check(y, [0.7] * 12, temperature=[1e-6, 2e-6, 1e-3, 0.05, 1e3, 1e30, 3e38, 1.0, 1.0, 1.0, 1.0, 1.0], least=12)


@pytest.mark.parametrize("size", [1.0, 1e-30, 1e6, 1e37])
def test_temperatures_of_all_magnitudes(size):
    """From one that leaves a single token to one that makes all alike, over logits of all sizes;
    the smallest is 2^-20, where neighbouring FP32 logits of 10 are an octave apart."""
    say("sample temperatures", size)
    g = np.random.default_rng(41)
    t = [float("inf"), 3e38, 1e30, 1e6, 50.0, 1.0, 0.02, 1e-3, 2.0 ** -19, 2.0 ** -20]
    y = logits(g, len(t), 9001, 2.0) * size
    y[:, 17::5] = -float("inf")
    for kw in ({}, dict(top_k=[700] * len(t)), dict(top_p=[0.7] * len(t)), dict(min_p=[0.3] * len(t)),
               dict(top_k=[8500] * len(t), top_p=[0.9] * len(t), min_p=[1e-3] * len(t))):
        check(y, g.random(len(t)), t, **kw)
    greedy, _ = lowbit.lowbit_sample(y, dev(g.random(len(t))), dev([0.0, -1.0, float("nan"), 9e-7, -0.0] * 2))
    assert np.array_equal(greedy.cpu().numpy(), y.cpu().numpy().argmax(1))


@pytest.mark.parametrize("n", [5, 5000, 151936])
def test_what_is_not_finite(n):
    say("sample not finite", n)
    g = np.random.default_rng(n)
    b = 8
    y = logits(g, b, n, 3.0)
    inf, nan = float("inf"), float("nan")
    y[0] = -inf
    y[1, :] = -inf
    y[1, n // 2] = 3.0
    y[2, n - 1] = nan
    y[2, 1] = inf
    y[3, 2], y[3, n - 1] = inf, inf
    y[4, ::2] = -inf
    y[5] = -3e38
    y[6, n - 2] = 3e38
    y[7, :3] = nan
    idx = check(y, g.random(b), [1.0, 0.7, 1.0, 0.5, 0.9, 1.0, 1.0, 1.0], top_k=[0, 3, 0, 2, 0, 0, 7, 1], least=7)
    assert idx.tolist()[:4] == [-1, n // 2, n - 1, 2] and idx[4] % 2 == 1 and idx[6] == n - 2 and idx[7] == 0


def test_a_mask_of_the_lowest_value():
    """Rows masked by the type's lowest number, not by infinity."""
    import torch

    g = np.random.default_rng(2)
    for y in ("f32", "bf16", "f16"):
        yt = logits(g, 6, 20000, 2.0, y)
        low = torch.finfo(yt.dtype).min
        yt[:, 100:] = low
        yt[5] = low
        idx = check(yt, g.random(6), top_k=[0, 5, 0, 500, 20000, 0], top_p=[1.0, 1.0, 0.9, 1.0, 0.5, 1.0])
        assert (idx[:5] < 100).all()


def test_wide_gaps_between_parts():
    """Parts of a row whose largest values lie octaves apart, in either order."""
    g = np.random.default_rng(5)
    b, n = 8, 30000
    y = logits(g, b, n, 1.0)
    for i, gap in enumerate((0, 3, 15, 30, 44, 60, 200, 5000)):
        y[i] += -gap * dev(np.arange(n) // 4096 % 4)
        if i % 2:
            y[i] = y[i].flip(0)
    check(y, g.random(b))
    check(y, g.random(b), top_k=[3000, 9000, 5000, 100, 2500, 4000, 29000, 8000])
    check(y, g.random(b), top_p=[0.9, 0.99, 0.999, 0.5, 0.95, 0.9999, 0.7, 0.8])


def test_strided_rows_and_given_outputs():
    import torch

    g = np.random.default_rng(6)
    wide = logits(g, 5, 3001, 2.0, "bf16")
    y = wide[:, 7:2999]
    idx, prob = dev([9] * 5, "int32"), dev([9.0] * 5)
    ws = torch.full((lowbit.lowbit_sample_workspace_bytes(2992, 5),), 255, dtype=torch.uint8, device="cuda")
    got = check(y, g.random(5), top_k=[4, 0, 50, 0, 1], idx=idx, prob=prob, workspace=ws)
    assert np.array_equal(got, idx.cpu().numpy())
    one, p1 = lowbit.lowbit_sample(y[2], dev([0.4]))  # a row alone
    assert one.shape == (1,) and 0 < float(p1) <= 1


def test_the_largest_vocabulary_and_equal_bits():
    import torch

    say("sample largest")
    g = np.random.default_rng(7)
    y = logits(g, 3, 1 << 20, 1.0)
    check(y, [0.1, 0.5, 0.999999], top_k=[0, 700000, 0], top_p=[1.0, 0.9, 0.99])
    settings = dict(top_k=dev([0, 700000, 0], "int32"), top_p=dev([1.0, 0.9, 0.99]))
    a = lowbit.lowbit_sample(y, dev([0.2, 0.6, 0.3]), **settings)
    for _ in range(3):
        c = lowbit.lowbit_sample(y, dev([0.2, 0.6, 0.3]), **settings)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_many_draws_follow_the_probabilities():
    """A grid of random numbers gives every token its share, to one in the grid."""
    g = np.random.default_rng(11)
    b, n = 4000, 30
    y = logits(g, 1, n, 1.5).repeat(b, 1)
    u = ((np.arange(b) + 0.5) / b).astype(np.float32)
    idx, _ = lowbit.lowbit_sample(y, dev(u), top_p=dev([0.95] * b))
    v = y[0].double().cpu().numpy()
    w = np.exp(v - v.max())
    order = np.argsort(-v)
    before = np.concatenate([[0], np.cumsum(w[order])[:-1]])
    w[order[before >= np.float32(0.95) * w.sum()]] = 0
    share = np.bincount(idx.cpu().numpy(), minlength=n) / b
    assert np.abs(share - w / w.sum()).max() <= 1.0 / b + 1e-6
