"""Attention over the 4-bit cache on the GPU where the weights of a row lie far apart: one
token ahead of all others, in every kernel, with the work-groups' shares short and long."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say
from tests.plain64 import U, rounding
from tests.test_kv_gpu import dt, host, i32

pytestmark = pytest.mark.gpu

# What a weight may lose in FP16: half a step relative, or half of the least number where it is
# small.  The largest weight of whatever shares a maximum stands at 2^7 at least.
LEAST = 2.0 ** -25 / 2.0 ** 7


def expected(q, k, v, last, scale, out_dtype):
    """One row and KV head: q [group][d], k and v [n][d] -> out, lse and their bounds.

    As tests/plain64_block.py derives them: scores of d FP32 products and their scaling, the
    exponential's 2^-21, a weight's rounding to FP16; an error e of a weight moves the result by
    e |v - out|; the sums' own roundings."""
    k, v = k[:last + 1], v[:last + 1]
    s = q @ k.T * scale
    es = (np.abs(q) @ np.abs(k).T) * abs(scale) * (q.shape[1] + 4) * U + np.abs(s) * 4 * U
    p = np.exp(s - s.max(1, keepdims=True))
    total = p.sum(1, keepdims=True)
    o = p @ v / total
    e = p * (es + 2.0 ** -21 + 2.0 ** -11) + np.minimum(p, LEAST)
    depth = (len(k) / 32 + 600) * U
    err = (e @ np.abs(v) + e.sum(1, keepdims=True) * np.abs(o)) / total * 1.01 + depth * 2 * (p @ np.abs(v)) / total
    lse = s.max(1) + np.log(total[:, 0])
    lbound = e.sum(1) / total[:, 0] * 1.01 + depth + 2.0 ** -20 + np.abs(lse) * 4 * U
    return o, lse, err + rounding(np.abs(o) + err, out_dtype), lbound


class Flat:
    """A cache of n tokens with keys of 0, but for those of `ahead`, whose keys have 8 in front
    (times what they are given) and whose values are 0."""

    def __init__(self, n, heads, d, page, ahead, seed=0):
        import torch

        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.heads, self.d, self.page = n, heads, d, page
        count = -(-n // page)
        self.pages = torch.zeros(count, P.page_bytes(heads, d, page), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(count, generator=g, device="cuda").int()
        k, v = [], []
        for at in range(0, n, 32768):
            t = torch.arange(at, min(n, at + 32768), device="cuda")
            kk = torch.zeros(len(t), heads, d, device="cuda")
            vv = torch.randn(len(t), heads, d, generator=g, device="cuda") * 0.2 + 0.7
            for token, f in ahead.items():
                if at <= token < at + len(t):
                    kk[token - at, :, 0], vv[token - at] = 8.0 * f, 0.0
            slots = (self.table[t // page] * page + t % page).int()
            lowbit.lowbit_kv_store(kk, vv, slots, self.pages, page)
            held = lowbit.lowbit_kv_load(self.pages, page, slots, heads, d)
            k.append(host(held[0]))
            v.append(host(held[1]))
        self.k, self.v = np.concatenate(k), np.concatenate(v)

    def run(self, octaves, b, nq, group, x, check):
        """b sequences that share the cache, each with nq queries whose scores of a token
        ahead are `octaves` in turn; those of `check` rows against 64 bits."""
        import torch

        hq, scale = self.heads * group, self.d ** -0.5
        q = torch.zeros(b * nq, hq, self.d, device="cuda")
        at = torch.arange(b * nq * hq, device="cuda").reshape(b * nq, hq) % len(octaves)
        q[:, :, 0] = torch.tensor(octaves, device="cuda")[at] * (np.log(2.0) / 8.0 / scale)
        q = q.to(dt(x))
        lse = torch.zeros(b * nq, hq, device="cuda")
        out = lowbit.lowbit_attention(q, self.pages, self.page, self.table.repeat(b, 1), i32([self.n] * b),
                                      q_start=i32(np.arange(b + 1) * nq), max_q=nq, scale=scale, lse=lse)
        got, glse, qv = host(out), host(lse), host(q)
        for row in np.unique(np.linspace(0, b * nq - 1, check).astype(int)):
            for h in range(self.heads):
                own = slice(h * group, (h + 1) * group)
                o, l, bound, lbound = expected(qv[row, own], self.k[:, h], self.v[:, h], self.n - nq + row % nq, scale,
                                               str(out.dtype).replace("torch.", ""))
                off = np.abs(got[row, own] - o)
                assert (off <= bound).all(), (row, h, octaves, float((off / bound).max()), float((off / np.abs(o)).max()))
                assert (np.abs(glse[row, own] - l) <= lbound).all(), (row, h)


OCTAVES = [23.0, 24.4, 25.1, 26.0, 22.0, 30.0]
# heads of d, queries of a KV head's group, rows of a sequence: each kernel
SHAPES = [(128, 1, 1), (256, 2, 1), (64, 4, 2), (128, 8, 4), (256, 2, 10), (64, 4, 12), (128, 4, 16), (128, 1, 100), (256, 1, 100),
          (64, 2, 70)]


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("d,group,nq", SHAPES)
def test_one_token_ahead_of_a_flat_rest(d, group, nq, x):
    """As many items as there are work-groups, so that a wave goes through thousands of tokens by
    one maximum; the token ahead first, in the middle, among the last."""
    say("attention ahead", d, group, nq, x)
    for first in (0, 7000, 15890):
        c = Flat(16000, 2, d, 64, {first: 1.0})
        c.run(OCTAVES, 300, nq, group, x, 3)


@pytest.mark.parametrize("d,group,nq", [(256, 6, 1), (128, 2, 1), (128, 1, 100), (256, 2, 40)])
def test_one_token_ahead_of_262143(d, group, nq):
    say("attention ahead of 262143", d, group, nq)
    c = Flat(262144, 1, d, 64, {3: 1.0})
    c.run([22.25, 24.6, 25.1, 17.0, 28.0, 20.0], 1, nq, group, "f16", 3)


@pytest.mark.parametrize("d,group,nq", SHAPES)
def test_maxima_that_rise_by_steps(d, group, nq):
    """Tokens ahead one after another, each by less or more than what raises the maximum."""
    say("attention rising", d, group, nq)
    c = Flat(6000, 1, d, 32, {5: 0.1, 700: 0.2, 1500: 0.45, 2100: 0.5, 3300: 0.9, 4800: 1.0})
    c.run([3.0, 10.0, 15.0, 16.0, 29.0, 100.0], 520, nq, group, "f16", 3)
