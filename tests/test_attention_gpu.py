"""Attention over the 4-bit cache on the GPU against tests/plain64_block.py:
every kernel, head layouts, lengths, pages, masks, rows that see nothing."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say
from tests.test_kv_gpu import NAMES, dt, host, i32

pytestmark = pytest.mark.gpu


class Case:
    """Random pages of b sequences; queries of the last nq[i] tokens of each."""

    def __init__(self, lens, nq, hq, heads, d, page, x="f16", seed=0, sharp=1.0, spare_rows=0, spare_pages=2, offset=0.0):
        import torch

        g = np.random.default_rng(seed + 7 * d + hq)
        self.lens, self.nq, self.heads, self.d, self.page = lens, nq, heads, d, page
        need = [-(-max(n, 0) // page) for n in lens]
        total = max(1, sum(need)) + spare_pages
        t = torch.Generator(device="cuda").manual_seed(seed + 1)
        pages = torch.zeros(total, P.page_bytes(heads, d, page), dtype=torch.uint8, device="cuda")
        slots = torch.arange(total * page, dtype=torch.int32, device="cuda")
        for at in range(0, total * page, 32768):
            part = slots[at:at + 32768]
            k = torch.randn(len(part), heads, d, generator=t, device="cuda") + offset
            v = torch.randn(len(part), heads, d, generator=t, device="cuda") * 0.7 + 0.2
            lowbit.lowbit_kv_store(k, v, part, pages, page)
        self.pages = pages
        order = g.permutation(total)
        cap = max(need + [1]) + 1
        self.table = np.full((len(lens), cap), -1, np.int64)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.start = np.concatenate([[0], np.cumsum(nq)])
        m = int(self.start[-1]) + spare_rows
        q = torch.randn(m, hq, d, generator=t, device="cuda") * sharp
        self.q = q.to(dt(x))
        self.scale = d ** -0.5

    def run(self, **kw):
        import torch

        one_each = all(n == 1 for n in self.nq) and self.q.shape[0] == len(self.nq) and not kw.pop("as_many", False)
        kw.pop("as_many", None)
        args = dict(q_start=None if one_each else i32(self.start), max_q=None if one_each else max(max(self.nq), 1),
                    scale=self.scale)
        args.update(kw)
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        out = lowbit.lowbit_attention(self.q, self.pages, self.page, i32(self.table), i32(self.lens), lse=lse, **args)
        return out, lse

    def kv(self, i):
        n = self.lens[i]
        t = np.arange(n)
        slots = self.table[i][t // self.page] * self.page + t % self.page
        return P.get(self.pages.cpu().numpy(), self.heads, self.d, self.page, slots)

    def check(self, out, lse, out_dtype=None, rows=None):
        """Sequences' rows (at most `rows` of each) against 64 bits."""
        got, glse, q = host(out), host(lse), host(self.q)
        name = str(out.dtype).replace("torch.", "")
        pages = self.pages.cpu().numpy()
        for i, (n, nq) in enumerate(zip(self.lens, self.nq)):
            t = np.arange(max(n, 0))
            slots = self.table[i][t // self.page] * self.page + t % self.page
            k, v = P.get(pages, self.heads, self.d, self.page, slots)
            pick = np.arange(nq) if rows is None or nq <= rows else np.unique(np.r_[0, nq - 1, np.linspace(0, nq - 1, rows).astype(int)])
            at = self.start[i] + pick
            want, wlse, bound, lbound = P.attention(q[at], k, v, n - nq + pick, self.scale, name)
            off = np.abs(got[at] - want)
            assert (off <= bound).all(), (i, n, nq, float((off / bound).max()))
            fine = np.isfinite(wlse)
            assert np.array_equal(np.isneginf(glse[at]), ~fine)
            assert (np.abs(glse[at] - wlse)[fine] <= lbound[fine]).all(), i


ONE = [(1, 16, 8, 128, 16), (1, 24, 4, 256, 64), (1, 1, 1, 64, 16), (2, 12, 4, 64, 32), (3, 32, 2, 128, 128), (2, 64, 1, 128, 16),
       (5, 40, 8, 128, 256), (1, 34, 2, 256, 32), (2, 33, 1, 64, 16), (1, 300, 1, 128, 16), (1, 7, 7, 256, 16)]


@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("b,hq,heads,d,page", ONE)
def test_one_token_of_each(x, b, hq, heads, d, page):
    say("attention one", x, b, hq, heads, d, page)
    for seed, lens in enumerate(([1, 17, 300, 15, 64], [2, 128, 16, 33, 500], [129, 31, 1, 700, 32])):
        c = Case(lens[:b], [1] * b, hq, heads, d, page, x, seed)
        out, lse = c.run()
        c.check(out, lse)


MANY = [  # lens, nq, hq, heads, d, page
    ([40], [5], 4, 1, 128, 16), ([40, 9, 300], [3, 9, 1], 8, 2, 64, 32), ([200], [7], 12, 4, 256, 16),
    ([70, 33], [8, 0], 16, 4, 128, 16), ([100], [16], 4, 1, 64, 16), ([130, 50], [30, 50], 6, 2, 128, 64),
    ([300], [300], 4, 1, 128, 16), ([257, 64, 1], [100, 64, 1], 8, 2, 256, 32), ([500], [129], 7, 1, 64, 16),
    ([90], [90], 3, 3, 64, 16), ([600], [260], 2, 2, 128, 128), ([20], [20], 260, 1, 64, 16), ([333], [333], 5, 1, 256, 16),
    ([64, 64], [40, 64], 32, 8, 128, 16)]


@pytest.mark.parametrize("x,out", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("lens,nq,hq,heads,d,page", MANY)
def test_several_tokens_of_each(x, out, lens, nq, hq, heads, d, page):
    say("attention many", x, out, lens, nq, hq, heads, d, page)
    c = Case(lens, nq, hq, heads, d, page, x, 3)
    o, lse = c.run(out_dtype=dt(out))
    c.check(o, lse)


@pytest.mark.parametrize("nq,max_q", [(1, 1), (1, 3), (1, 40), (1, 1000), (5, 1), (5, 8), (40, 2), (40, 500)])
def test_any_promise_of_the_most_rows(nq, max_q):
    """max_q picks the kernel; the result does not go by it."""
    say("attention max_q", nq, max_q)
    c = Case([77, 300, nq], [nq] * 3, 12, 4, 128, 16, seed=nq)
    out, lse = c.run(as_many=True, max_q=max_q)
    c.check(out, lse)


@pytest.mark.parametrize("hq,heads,d,nq", [(24, 4, 256, 1), (16, 8, 128, 1), (8, 2, 64, 4), (32, 8, 128, 70), (12, 4, 256, 40)])
def test_rows_that_see_nothing_and_rows_of_no_sequence(hq, heads, d, nq):
    import torch

    say("attention empty", hq, heads, d, nq)
    # no tokens at all; fewer tokens than queries; no queries; a negative length; one token
    lens, nqs = [0, max(nq // 2, 0), 50, -3, nq + 1], [nq, nq, 0, nq, nq]
    c = Case([max(n, 0) for n in lens], nqs, hq, heads, d, 16, seed=5, spare_rows=6)
    c.lens = lens
    out = torch.full(c.q.shape, 3.0, dtype=c.q.dtype, device="cuda")
    _, lse = c.run(out=out)
    c.lens = [max(n, 0) for n in lens]
    c.check(out, lse)
    assert (out[-6:] == 3.0).all() and (lse[-6:] == 7.0).all()
    assert not out[:nq].any() and torch.isneginf(lse[:nq]).all()


def test_lengths_past_the_table_are_cut():
    c = Case([40], [1], 8, 2, 128, 16)
    table = c.table[:, :3]  # 48 tokens, of which the last page is full
    c.table, c.lens = table, [48]
    want, wlse = c.run()
    c.lens = [2 ** 31 - 1]
    got, lse = c.run()
    import torch

    assert torch.equal(got, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("nq,d,hq,heads", [(1, 128, 8, 2), (20, 128, 8, 2), (100, 64, 4, 1), (1, 256, 24, 4), (60, 256, 2, 1)])
def test_pages_that_are_not_there_are_masked(nq, d, hq, heads):
    say("attention absent pages", nq, d)
    c = Case([400], [nq], hq, heads, d, 16, seed=2)
    gone = [0, 3, 4, 11, 24]
    bad = c.table.copy()
    bad[0, gone] = [-1, c.pages.shape[0], 2 ** 31 - 1, -2 ** 31, -7]
    keep = c.table
    c.table = bad
    out, lse = c.run()
    # the same from the tokens that are left, rows by their last token
    t = np.array([i for i in range(400) if i // 16 not in gone])
    k, v = P.get(c.pages.cpu().numpy(), heads, d, 16, keep[0][t // 16] * 16 + t % 16)
    last = np.array([int((t <= 400 - nq + j).sum()) - 1 for j in range(nq)])
    want, wlse, bound, lbound = P.attention(host(c.q), k, v, last, c.scale, "float16")
    assert (np.abs(host(out) - want) <= bound).all() and (np.abs(host(lse) - wlse) <= lbound).all()
    # none of them there
    c.table = np.full_like(keep, -1)
    out, lse = c.run()
    assert not out.any() and np.isneginf(host(lse)).all()


@pytest.mark.parametrize("nq,d", [(1, 64), (1, 128), (1, 256), (9, 128), (100, 128), (100, 256), (40, 64)])
def test_what_lies_behind_the_last_token_does_not_matter(nq, d):
    """Bytes of the last page past the length, and of pages behind it, that stand
    for infinities and NaN."""
    import torch

    c = Case([133], [nq], 4, 2, d, 64, seed=1)
    want, wlse = c.run()
    c.table[0, 3] = c.free[0]
    c.pages[int(c.free[0])] = 255
    page = c.pages[int(c.table[0, 2])].view(2, -1)  # tokens 128..132 are there, 133.. are not
    g, size = d // 32, 64 * d // 2
    page[:, :size].view(2, 64, -1)[:, 5:] = 255
    page[:, size:size + 64 * g * 4].view(2, 64, -1)[:, 5:] = 255
    base = size + 64 * g * 4
    vc = page[:, base:base + size].view(2, 16, d // 2, 4)
    vc[:, 2:] = 255
    vc[:, 1, :, [2, 1, 3]] = 255  # tokens 5, 6, 7
    vp = page[:, base + size:].view(2, 16, g, 2, 4, 2)
    vp[:, 2:] = 255
    vp[:, 1, :, :, 1:] = 255
    got, lse = c.run()
    assert torch.equal(got, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("sharp,offset", [(0.0, 0.0), (1e-6, 0.0), (30.0, 0.0), (400.0, 0.0), (3.0, 40.0)])
@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("nq", [1, 70])
def test_flat_and_sharp_scores(sharp, offset, x, nq):
    """All scores alike, one that takes all, and maxima that rise on the way."""
    say("attention scores", sharp, offset, x, nq)
    c = Case([700], [nq], 4, 1, 128, 16, x, seed=4, sharp=sharp, offset=offset)
    out, lse = c.run()
    c.check(out, lse, rows=12)


def test_queries_of_all_magnitudes():
    import torch

    c = Case([200] * 9, [1] * 9, 4, 2, 128, 16, "bf16", seed=6)
    for i, f in enumerate((1e-38, 1e-30, 1e-12, 1e-4, 1.0, 1e3, 1e10, 1e20, 0.0)):
        c.q[i] *= f
    c.q[8, 0, 5] = 2e-39
    c.scale = 1e-3
    out, lse = c.run()
    got = host(out)
    assert np.isfinite(got).all()
    for i in (0, 1, 2, 3, 4, 5, 8):  # the larger ones' scores pass FP32's exact range
        k, v = c.kv(i)
        want, wlse, bound, lbound = P.attention(host(c.q)[i:i + 1], k, v, [199], c.scale, "bfloat16")
        assert (np.abs(got[i:i + 1] - want) <= bound).all() and (np.abs(host(lse)[i:i + 1] - wlse) <= lbound).all()
    # a query that is not finite spoils its own head alone
    c = Case([50, 60], [1, 1], 4, 2, 128, 16, "f16", seed=6)
    want, _ = c.run()
    c.q[0, 1, 3], c.q[1, 2, 0] = float("nan"), float("inf")
    got, _ = c.run()
    bad = torch.isnan(got)
    assert bad[0, 1].all() and bad[1, 2].all() and int(bad.sum()) == 2 * 128
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("lens,hq,heads,d,page", [([20000, 3, 5000], 24, 4, 256, 64), ([70001], 8, 8, 128, 16), ([33000], 64, 1, 64, 256),
                                                  ([9000, 8999, 1, 12345], 16, 2, 128, 32)])
def test_long_contexts(lens, hq, heads, d, page):
    say("attention long", lens, hq, heads, d, page)
    c = Case(lens, [1] * len(lens), hq, heads, d, page, seed=8)
    out, lse = c.run()
    c.check(out, lse)


def test_a_long_chunk():
    say("attention chunk")
    c = Case([5000, 1500], [1100, 1500], 8, 2, 128, 16, "bf16", seed=9)
    out, lse = c.run()
    c.check(out, lse, rows=9)


def test_many_sequences():
    g = np.random.default_rng(1)
    say("attention many sequences")
    for b in (300, 1100):
        lens = [int(v) for v in g.integers(1, 60, b)]
        c = Case(lens, [1] * b, 4, 1, 64, 16, seed=b)
        out, lse = c.run()
        c.check(out, lse)


def test_strides_and_heads_first():
    import torch

    c = Case([100, 37], [20, 3], 8, 2, 128, 16, "f16", seed=3)
    want, _ = c.run()
    m = c.q.shape[0]
    wide = torch.zeros(m, 12, 137, dtype=torch.float16, device="cuda")
    wide[:, 2:10, 5:133] = c.q
    tables = torch.full((2, 40), -9, dtype=torch.int32, device="cuda")
    tables[:, 3:3 + c.table.shape[1]] = i32(c.table)
    out = torch.zeros(8, m, 130, dtype=torch.float16, device="cuda")
    got = lowbit.lowbit_attention(wide[:, 2:10, 5:133], c.pages, 16, tables[:, 3:3 + c.table.shape[1]], i32(c.lens),
                                  q_start=i32(c.start), max_q=20, scale=c.scale, out=out[:, :, 1:129].transpose(0, 1))
    assert torch.equal(got, want) and not out[:, :, 0].any() and not out[:, :, 129].any()
    # d^-0.5 and m rows where nothing is said
    got = lowbit.lowbit_attention(c.q, c.pages, 16, i32(c.table), i32(c.lens), q_start=i32(c.start))
    c.check(got, c.run()[1])


def test_equal_inputs_equal_bits_whatever_the_workspace_held():
    import torch

    for nq in (1, 6, 90):
        c = Case([3000, 700], [nq] * 2, 8, 2, 128, 16, seed=nq)
        need = lowbit.lowbit_attention_workspace_bytes(2 * nq, 2, 8, 2, 128, nq)
        first = None
        for fill in (0, 255, 127):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            out, lse = c.run(workspace=ws)
            first = first or (out, lse)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_broken_row_limits_stay_inside():
    """q_start that is no ascending list names rows that are there or none."""
    import torch

    c = Case([50] * 3, [2, 2, 2], 4, 1, 64, 16, seed=1, spare_rows=2)
    for start in ([0, 9, 2, 100], [-5, -1, 3, 2 ** 31 - 1], [8, 6, 4, 2], [-2 ** 31, 0, 0, 0]):
        out, _ = c.run(q_start=i32(start), max_q=2)
        torch.cuda.synchronize()
        assert out.shape == c.q.shape
