"""The plain forms of tests/plain64_block.py held to values worked out by hand
and to plain loops."""
import math

import numpy as np

from tests import plain64_block as P


def test_rotary_by_hand():
    quarter = 2 ** 62  # a quarter of a turn a position
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    for pos, half, inter in ((0, [1, 2, 3, 4], [1, 2, 3, 4]), (1, [-3, -4, 1, 2], [-2, 1, -4, 3]),
                             (2, [-1, -2, -3, -4], [-1, -2, -3, -4]), (-1, [3, 4, -1, -2], [2, -1, 4, -3]),
                             (2 ** 31 - 1, [3, 4, -1, -2], [2, -1, 4, -3])):
        assert np.allclose(P.rope(x, [pos], [quarter] * 2), half, atol=1e-6)
        assert np.allclose(P.rope(x, [pos], [quarter] * 2, interleaved=True), inter, atol=1e-6)
    out = P.rope(x, [1], [quarter], gain=0.5)  # half of the head turns
    assert np.allclose(out, [-1.0, 0.5, 3, 4], atol=1e-6)


def test_frequencies_by_hand():
    f, gain = P.frequencies(4, 10000.0)
    assert np.allclose(f, [1.0, 0.01]) and gain == 1.0
    assert np.allclose(P.frequencies(4, 10000.0, "linear", 8.0)[0], [0.125, 0.00125])
    assert np.allclose(P.frequencies(4, 10000.0, "ntk", 4.0)[0], [1.0, (10000.0 * 16) ** -0.5])
    # 64 values, theta 10000, trained at 4096: pairs below the eleventh stay, those from the 23rd on are divided
    f, gain = P.frequencies(64, 10000.0, "yarn", 16.0, 4096)
    plain = P.frequencies(64, 10000.0)[0]
    lo = math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000.0)))
    hi = math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000.0)))
    assert (lo, hi) == (10, 23)
    assert np.allclose(f[:11], plain[:11]) and np.allclose(f[23:], plain[23:] / 16)
    assert all(plain[i] / 16 < f[i] < plain[i] for i in range(11, 23))
    assert abs(gain - (0.1 * math.log(16) + 1)) < 1e-15


def test_codes_by_hand():
    # 0, 1, .. 15 twice: a = 16, b = -16, the codes are the numbers
    x = np.tile(np.arange(16, dtype=np.float32), 2)
    code, a, b = P.quantise(x)
    assert a == 16 and b == -16 and np.array_equal(code, x.astype(np.uint8))
    assert np.array_equal(P.dequantise(code, a, b), x.astype(np.float16))
    # ties to even: half a step above an even and an odd code
    x[3], x[5], x[20] = 2.5, 5.5, 14.5
    code, a, b = P.quantise(x)
    assert (code[3], code[5], code[20]) == (2, 6, 14)
    # one value everywhere: a = 0
    code, a, b = P.quantise(np.full(32, 0.3, np.float32))
    assert a == 0 and not code.any() and P.dequantise(code, a, b)[0] == np.float16(0.3)
    # nothing that is not finite is held
    x = np.zeros(32, np.float32)
    x[:3] = np.nan, np.inf, -np.inf
    v = P.held(x)
    assert np.isfinite(v).all() and abs(v[1] - 16384) <= 1200 and abs(v[2] + 16384) <= 1200
    g = np.random.default_rng(3)
    for sigma in (1e-6, 1e-3, 1.0, 300.0, 1e5):
        x = (g.standard_normal((50, 64)) * sigma).astype(np.float32)
        assert (np.abs(P.held(x).astype(np.float64) - np.clip(x, -16384, 16384)) <= P.held_bound(x)).all()


def test_pages_by_hand_and_back():
    heads, d, page = 2, 64, 16
    g = np.random.default_rng(4)
    pages = np.zeros((3, P.page_bytes(heads, d, page)), np.uint8)
    k, v = (g.standard_normal((5, heads, d)).astype(np.float32) for _ in range(2))
    slots = [5, 47, 16, -1, 48]
    P.put(pages, heads, d, page, slots, k, v)
    kk, vv = P.get(pages, heads, d, page, slots)
    for i in range(3):
        assert np.array_equal(kk[i], P.held(k[i])) and np.array_equal(vv[i], P.held(v[i]))
    assert not kk[3:].any() and not vv[3:].any()
    # token 5 of page 0, head 1: K codes, its params, V bytes (token 1 of the second four is byte 2)
    part = pages[0].reshape(heads, -1)[1]
    code, a, b = P.quantise(k[0, 1].reshape(2, 32))
    assert part[5 * 32 + 7] == code[0, 14] | (code[0, 15] << 4)
    assert np.array_equal(part[16 * 32 + 5 * 8:16 * 32 + 6 * 8].copy().view(np.float16), [a[0], b[0], a[1], b[1]])
    code, a, b = P.quantise(v[0, 1].reshape(2, 32))
    base = 16 * 32 + 16 * 8
    assert part[base + (32 + 20) * 4 + 2] == code[1, 8] | (code[1, 9] << 4)
    q = part[base + 16 * 32:].copy().view(np.float16).reshape(4, 2, 2, 4)
    assert q[1, 1, 0, 1] == a[1] and q[1, 1, 1, 1] == b[1]


def test_attention_by_hand():
    # one head, two tokens whose scores differ by ln 3: weights 1/4 and 3/4
    q = np.array([[[math.log(3.0), 0.0]]])
    k = np.array([[[0.0, 1.0]], [[1.0, 1.0]]])
    v = np.array([[[4.0, 0.0]], [[8.0, 1.0]]])
    out, lse, bound, _ = P.attention(q, k, v, [1], 1.0, "float32")
    assert np.allclose(out, [[[7.0, 0.75]]]) and np.allclose(lse, math.log(4.0)) and (bound < 0.03).all()
    out, lse, _, _ = P.attention(q, k, v, [0], 1.0, "float32")
    assert np.allclose(out, [[[4.0, 0.0]]]) and np.allclose(lse, 0.0)
    out, lse, _, _ = P.attention(q, k, v, [-1], 1.0, "float32")
    assert not out.any() and np.isneginf(lse).all()


def test_sampling_by_hand():
    # weights 4, 2, 1, 1 in the order of their values; by number: 1, 4, 1, 2
    y = np.log(np.array([1.0, 4.0, 1.0, 2.0]))
    pick = lambda u, **k: P.sample(y, u, **k)[:2]  # noqa: E731
    for u, token, p in ((0.0, 0, 1 / 8), (0.12, 0, 1 / 8), (0.13, 1, 0.5), (0.62, 1, 0.5), (0.63, 2, 1 / 8), (0.76, 3, 0.25),
                        (2.0, 3, 0.25), (-1.0, 0, 1 / 8), (float("nan"), 0, 1 / 8)):
        got = pick(u)
        assert got[0] == token and abs(got[1] - p) < 1e-12
    assert pick(0.9, top_k=1) == (1, 1.0)
    assert pick(0.1, top_k=3) == (0, pick(0.1, top_k=3)[1])  # of two equal ones the lower number stays
    assert pick(0.7, top_k=2)[0] == 3 and abs(pick(0.7, top_k=2)[1] - 1 / 3) < 1e-12
    assert pick(0.99, top_p=0.4) == (1, 1.0) and pick(0.99, top_p=0.6)[0] == 3 and pick(0.99, top_p=0.0) == (1, 1.0)
    assert pick(0.0, min_p=0.6) == (1, 1.0) and pick(0.0, min_p=0.3)[0] == 1
    assert pick(0.0, min_p=7.0) == (1, 1.0)
    assert pick(0.5, temperature=0.0) == (1, 1.0) and pick(0.5, temperature=float("nan")) == (1, 1.0)
    # temperature 1/2 squares the weights: 1, 16, 1, 4
    assert abs(P.sample(y, 0.5, temperature=0.5)[1] - 16 / 22) < 1e-7
    assert P.sample(np.array([-np.inf, -np.inf]), 0.5)[0] == -1
    assert P.sample(np.array([1.0, np.nan, np.inf]), 0.5)[:2] == (1, 1.0)
    assert P.sample(np.array([1.0, np.inf, np.inf]), 0.9)[:2] == (1, 1.0)
