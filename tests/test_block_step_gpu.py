"""A decode step with its attention and its draw, as it is put together from the
library's calls: embedding gather, norm, the fused Q / K / V product, keys into the
4-bit cache and queries turned beside them, attention, output product, norm and
residual, LM head, penalties, a token drawn from each row.

Each stage is held to the 64-bit oracle on the inputs it got.  The matrices
are small enough for the GEMV that has no atomics, so the step is a function of
its inputs: captured in a graph and replayed, it has to give the same bits as
eager calls, token after token.
"""
import numpy as np
import pytest

import oracle
from bit_matmul_lowbit_amd import lowbit, synth
from tests import plain64_block as P
from tests.helpers import assert_close, dev_u16, host_u16, say
from tests.test_kv_gpu import host

pytestmark = pytest.mark.gpu

B, K, HQ, KV, D, PAGE, VOCAB, CAP = 6, 512, 8, 2, 64, 16, 5003, 8
ROT = 32


class Block:
    """A block of a model and what a serving program keeps: pages and their table, lengths,
    workspaces, outputs, each request's settings.  Request 4 has no place in the batch."""

    def __init__(self, fmt, seed):
        import torch

        self.fmt, g = fmt, synth.rng(seed)
        f32 = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.host = {}
        for name, n, k in (("embed", VOCAB, K), ("qkv", (HQ + 2 * KV) * D, K), ("o", K, HQ * D), ("head", VOCAB, K)):
            if fmt == "q1":
                c, s = oracle.q1_quantize(synth.fp16_normal(g, (n, k), 0.1))
            else:
                c, s = oracle.t2_pack(synth.ternary(g, (n, k)), synth.fp16_uniform(g, (n, k // 128), 0.01, 0.1))
            self.host[name] = (c, s, n, k)
            setattr(self, name, (torch.from_numpy(c).cuda(), dev_u16(s), n, k))
        self.w = [1 + f32(K) / 8 for _ in range(2)]
        self.turns, self.gain = lowbit.lowbit_rope_turns(ROT, 1e6, "yarn", 4.0, 64)
        n_pages = B * CAP + 3
        self.pages = torch.zeros(n_pages, lowbit.lowbit_kv_page_bytes(KV, D, PAGE), dtype=torch.uint8, device="cuda")
        self.table = torch.from_numpy(g.permutation(n_pages)[:B * CAP].reshape(B, CAP).astype(np.int32)).cuda()
        self.start = [14, 1, 40, 31, 0, 95]  # tokens in the cache before the first step
        self.live = torch.tensor([n > 0 for n in self.start], device="cuda")
        for i, n in enumerate(self.start):
            if n:
                t = torch.arange(n, device="cuda")
                slots = (self.table[i][t // PAGE] * PAGE + t % PAGE).int()
                lowbit.lowbit_kv_store(f32(n, KV, D), f32(n, KV, D), slots, self.pages, PAGE, t.int(), self.turns)
        self.pages0 = self.pages.clone()
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.length, self.last = e(B, dtype=torch.int32), e(B, dtype=torch.int32)
        self.emb, self.x0, self.x1 = (e(B, K, dtype=torch.float16) for _ in range(3))
        self.fused, self.r0, self.r1, self.y = e(B, (HQ + 2 * KV) * D), e(B, K), e(B, K), e(B, K)
        self.q, self.att = (e(B, HQ, D, dtype=torch.float16) for _ in range(2))
        self.slots = e(B, dtype=torch.int32)
        self.logits, self.out = e(B, VOCAB), e(B, VOCAB)
        self.idx, self.prob, self.u = e(B, dtype=torch.int32), e(B), e(B)
        self.u_steps = torch.rand(16, B, generator=torch.Generator().manual_seed(seed)).cuda()
        self.bias_ids = torch.from_numpy(g.integers(0, VOCAB, (B, 6)).astype(np.int32)).cuda()
        self.bias_vals = f32(B, 6) * 3
        self.settings = [torch.tensor(v, dtype=t, device="cuda") for v, t in (
            ([0.5, 1.0, 0.0, 1.3, 1.0, 0.8], torch.float32), ([20, 0, 0, 0, 5, 300], torch.int32),
            ([0.85, 1.0, 1.0, 0.9, 1.0, 0.95], torch.float32), ([0.0, 0.02, 0.0, 0.0, 0.1, 0.0], torch.float32))]
        need = max([lowbit.lowbit_gemv_workspace_bytes(fmt, n, k, B) for _, _, n, k in self.host.values()]
                   + [lowbit.lowbit_logits_workspace_bytes(VOCAB, B), lowbit.lowbit_sample_workspace_bytes(VOCAB, B),
                      lowbit.lowbit_attention_workspace_bytes(B, B, HQ, KV, D)])
        self.ws = e(need, dtype=torch.uint8)  # one for all calls of the stream
        self.reset()

    def reset(self):
        import torch

        self.pages.copy_(self.pages0)
        self.length.copy_(torch.tensor(self.start, dtype=torch.int32))
        self.last.copy_(torch.arange(B, dtype=torch.int32) * 700 + 5)

    def project(self, name, x, y):
        c, s, n, k = getattr(self, name)
        lowbit.lowbit_gemv(self.fmt, c, s, n, k, x, out=y, workspace=self.ws)

    def step(self):
        import torch

        c, s, n, k = self.embed
        lowbit.lowbit_embed(self.fmt, c, s, n, k, self.last, out=self.emb)
        self.r0.copy_(self.emb)
        lowbit.lowbit_norm_residual(None, self.r0, pre="rms", pre_w=self.w[0], x_out=self.x0)
        self.project("qkv", self.x0, self.fused)
        position = self.length.long()
        page = self.table.gather(1, (position // PAGE).unsqueeze(1)).squeeze(1).long()
        self.slots.copy_(torch.where(self.live, page * PAGE + position % PAGE, -1))
        heads = self.fused.view(B, HQ + 2 * KV, D)
        lowbit.lowbit_kv_store(heads[:, HQ:HQ + KV], heads[:, HQ + KV:], self.slots, self.pages, PAGE, self.length,
                               self.turns, gain=self.gain, q=heads[:, :HQ], q_out=self.q)
        self.length.add_(self.live)
        lowbit.lowbit_attention(self.q, self.pages, PAGE, self.table, self.length, out=self.att, workspace=self.ws)
        self.project("o", self.att.view(B, HQ * D), self.y)
        lowbit.lowbit_norm_residual(self.y, self.r0, pre="rms", pre_w=self.w[1], r_out=self.r1, x_out=self.x1)
        self.project("head", self.x1, self.logits)
        lowbit.lowbit_logits_process(self.logits, bias_ids=self.bias_ids, bias_vals=self.bias_vals, out=self.out,
                                     top1=False, workspace=self.ws)
        lowbit.lowbit_sample(self.out, self.u, *self.settings, idx=self.idx, prob=self.prob, workspace=self.ws)
        self.last.copy_(self.idx)


def _check_stages(m, pages_before, position):
    of = oracle.Q1 if m.fmt == "q1" else oracle.T2
    for name, x, y in (("qkv", m.x0, m.fused), ("o", m.att.view(B, HQ * D), m.y), ("head", m.x1, m.logits)):
        c, s, n, k = m.host[name]
        assert_close(y.cpu().double().numpy(), oracle.gemv(of, c, s, n, k, host_u16(x)), name)
    # the cache: V as it is, K held within what its rounding and that of the turning may cost
    fused = m.fused.cpu().numpy().reshape(B, HQ + 2 * KV, D)
    turns, slots, live = m.turns.cpu().numpy(), m.slots.cpu().numpy(), m.live.cpu().numpy()
    assert (slots[~live] == -1).all() and (slots[live] >= 0).all()
    held_k, held_v = P.get(m.pages.cpu().numpy(), KV, D, PAGE, slots)
    assert np.array_equal(held_v[live], P.held(fused[:, HQ + KV:])[live])
    x = fused[:, HQ:HQ + KV]
    turned = P.rope(x, position, turns, False, m.gain)
    err = P.rope_bound(x, position, turns, False, m.gain, "float32").max(-1, keepdims=True)
    bound = P.held_bound(turned.astype(np.float32)) + 2 * err
    assert (np.abs(held_k.astype(np.float64) - turned) <= bound)[live].all()
    x = fused[:, :HQ]
    q = P.rope(x, position, turns, False, m.gain)
    assert (np.abs(host(m.q) - q) <= P.rope_bound(x, position, turns, False, m.gain, "float16")).all()
    # nothing but the slots' own bytes
    want = pages_before.copy()
    P.put(want, KV, D, PAGE, slots, np.zeros((B, KV, D), np.float32), np.zeros((B, KV, D), np.float32))
    now = m.pages.cpu().numpy().copy()
    P.put(now, KV, D, PAGE, slots, np.zeros((B, KV, D), np.float32), np.zeros((B, KV, D), np.float32))
    assert np.array_equal(now, want)
    # attention over what the cache holds
    table, length = m.table.cpu().numpy(), m.length.cpu().numpy()
    for i in range(B):
        t = np.arange(length[i])
        kk, vv = P.get(m.pages.cpu().numpy(), KV, D, PAGE, table[i][t // PAGE] * PAGE + t % PAGE)
        out, _, bound, _ = P.attention(host(m.q)[i:i + 1], kk, vv, np.array([length[i] - 1]), D ** -0.5, "float16")
        assert (np.abs(host(m.att)[i:i + 1] - out) <= bound).all(), i
    # the draw
    y, u = m.out.cpu().double().numpy(), m.u.cpu().numpy()
    t, k, p, mp = (s.cpu().numpy() for s in m.settings)
    for i in range(B):
        token, prob, margin = P.sample(y[i], u[i], t[i], k[i], p[i], mp[i])
        if margin > 2.0 ** -34:
            assert m.idx[i].item() == token and abs(m.prob[i].item() - prob) <= prob * 2.0 ** -22


@pytest.mark.parametrize("fmt", ["q1", "t2"])
def test_steps_eager_and_as_a_graph(fmt):
    import torch

    say("steps with attention and a draw", fmt)
    m = Block(fmt, 31)
    eager = []
    for i in range(10):  # request 0 goes on to its second page, 3 to its third, 5 to its seventh
        m.u.copy_(m.u_steps[i])
        before, position = m.pages.cpu().numpy(), m.length.cpu().numpy()
        m.step()
        torch.cuda.synchronize()
        _check_stages(m, before, position)
        eager.append([t.clone() for t in (m.idx, m.prob, m.att, m.r1, m.out, m.pages)])
    assert m.length.tolist() == [n + 10 if n else 0 for n in m.start]
    assert len({tuple(e[0].tolist()) for e in eager}) > 1
    m.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    m.reset()
    for i, want in enumerate(eager):
        for t in (m.q, m.att, m.fused, m.logits, m.out, m.r1, m.prob):
            t.fill_(3.0)
        m.ws.fill_(0x5A)
        m.u.copy_(m.u_steps[i])
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((m.idx, m.prob, m.att, m.r1, m.out, m.pages), want):
            assert torch.equal(t, w), i


def test_a_chunk_then_single_tokens_see_the_same_cache():
    """A prompt written and attended in one chunk, in two, or token by token: the same bytes
    in the cache, and rows that agree within FP16's rounding of what each computes."""
    import torch

    say("a prompt in chunks")
    g = torch.Generator(device="cuda").manual_seed(9)
    n, hq, heads, d, page = 150, 8, 2, 128, 32
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda") for h in (hq, heads, heads))
    turns, _ = lowbit.lowbit_rope_turns(d)
    table = torch.tensor([[4, 1, 0, 5, 2]], dtype=torch.int32, device="cuda")
    runs = []
    for cuts in ([0, n], [0, 67, n], list(range(n + 1))):
        pages = torch.zeros(6, lowbit.lowbit_kv_page_bytes(heads, d, page), dtype=torch.uint8, device="cuda")
        rows = []
        for lo, hi in zip(cuts, cuts[1:]):
            t = torch.arange(lo, hi, device="cuda")
            slots = (table[0][t // page] * page + t % page).int()
            qq = lowbit.lowbit_kv_store(k[lo:hi], v[lo:hi], slots, pages, page, t.int(), turns, q=q[lo:hi])
            length = torch.tensor([hi], dtype=torch.int32, device="cuda")
            start = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
            rows.append(lowbit.lowbit_attention(qq, pages, page, table, length, start, hi - lo, out_dtype=torch.float32)
                        if hi - lo > 1 else
                        lowbit.lowbit_attention(qq, pages, page, table, length, out_dtype=torch.float32))
        runs.append((pages, torch.cat(rows).double().cpu().numpy()))
    kk, vv = P.get(runs[0][0].cpu().numpy(), heads, d, page,
                   (table[0].repeat_interleave(page)[:n] * page + torch.arange(n, device="cuda") % page).cpu().numpy())
    rope = lowbit.lowbit_rope(q, torch.arange(n, dtype=torch.int32, device="cuda"), turns, out_dtype=torch.float16)
    out, _, bound, _ = P.attention(host(rope), kk, vv, np.arange(n), d ** -0.5, "float32")
    for pages, got in runs:
        assert torch.equal(pages, runs[0][0])
        assert (np.abs(got - out) <= bound).all()
