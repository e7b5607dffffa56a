"""A decode step as it is put together from the library's calls: embedding
gather, norm, projections with the requests' adapters beside them, the gated
product, norm and residual, LM head, penalties and grammar, the token.

Each stage is held to the 64-bit oracle on the inputs it got.  The matrices are
small enough for the GEMV that has no atomics, so the whole step is a function
of its inputs: captured in a graph and replayed, it has to give the same bits
as eager calls, token after token.
"""
import numpy as np
import pytest

import oracle
from bit_matmul_lowbit_amd import lowbit, synth
from tests import plain64
from tests.helpers import assert_close, dev_u16, host_u16, say

pytestmark = pytest.mark.gpu

B, K, F, VOCAB, SLOTS, R, CAP = 5, 512, 1024, 3001, 3, 16, 40


class Model:
    """One block with its embedding and head, and what a serving program keeps:
    adapters, workspaces, outputs, the requests' tokens."""

    def __init__(self, fmt, seed):
        import torch

        self.fmt, g = fmt, synth.rng(seed)
        f32 = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        f16 = lambda *s: f32(*s).half()  # noqa: E731
        self.host = {}
        for name, n, k in (("embed", VOCAB, K), ("gu", 2 * F, K), ("dn", K, F), ("head", VOCAB, K)):
            if fmt == "q1":
                c, s = oracle.q1_quantize(synth.fp16_normal(g, (n, k), 0.1))
            else:
                c, s = oracle.t2_pack(synth.ternary(g, (n, k)), synth.fp16_uniform(g, (n, k // 128), 0.01, 0.2))
            self.host[name] = (c, s, n, k)
            setattr(self, name, (torch.from_numpy(c).cuda(), dev_u16(s), n, k))
        self.adapters = {"gu": (f16(SLOTS, R, K) / 16, f16(SLOTS, 2 * F, R) / 8),
                         "dn": (f16(SLOTS, R, F) / 32, f16(SLOTS, K, R) / 8)}
        self.ids = torch.tensor([2, -1, 0, 2, 1], dtype=torch.int32, device="cuda")
        self.ranks = torch.tensor([16, 5, 9], dtype=torch.int32, device="cuda")
        self.scales = torch.tensor([1.0, 0.5, 2.0], device="cuda")
        self.w = [1 + f32(K) / 8 for _ in range(3)]
        self.gate = 1 + f32(B, K) / 8
        self.tokens = torch.from_numpy(g.integers(0, VOCAB, (B, CAP)).astype(np.int32)).cuda()
        self.tokens0 = self.tokens.clone()
        self.prompt_len = torch.tensor([3, 7, 1, 12, 5], dtype=torch.int32, device="cuda")
        self.total_len = self.prompt_len.clone()
        self.penalties = [torch.tensor(v, device="cuda") for v in
                          ([1.3, 1.0, 1.1, 2.0, 1.2], [0.2, 0.0, 0.5, 0.1, 0.0], [0.1, 0.4, 0.0, 0.2, 0.0])]
        self.mask = torch.from_numpy(g.integers(-2 ** 31, 2 ** 31, (2, (VOCAB + 31) // 32)).astype(np.int32)).cuda()
        self.mask_row = torch.tensor([0, -1, 1, 0, -1], dtype=torch.int32, device="cuda")
        self.bias_ids = torch.from_numpy(g.integers(0, VOCAB, (B, 6)).astype(np.int32)).cuda()
        self.bias_vals = f32(B, 6) * 3
        e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.h, self.y, self.logits, self.out = e(B, 2 * F), e(B, K), e(B, VOCAB), e(B, VOCAB)
        self.z, self.x0, self.x1 = (e(B, n, dtype=torch.float16) for n in (F, K, K))
        self.emb = e(B, K, dtype=torch.float16)
        self.r0, self.r1 = e(B, K), e(B, K)
        self.h0, self.y0 = e(B, 2 * F), e(B, K)
        self.idx, self.val = e(B, dtype=torch.int32), e(B)
        self.last = self.tokens[torch.arange(B), self.prompt_len.long() - 1].contiguous()
        self.last0 = self.last.clone()
        need = max([lowbit.lowbit_gemv_workspace_bytes(fmt, n, k, B) for _, _, n, k in self.host.values()]
                   + [lowbit.lowbit_lora_workspace_bytes(B, n, k, R, SLOTS) for n, k in ((2 * F, K), (K, F))]
                   + [lowbit.lowbit_logits_workspace_bytes(VOCAB, B)])
        self.ws = e(need, dtype=torch.uint8)  # one for all calls of the stream

    def project(self, name, x, y, before):
        c, s, n, k = getattr(self, name)
        lowbit.lowbit_gemv(self.fmt, c, s, n, k, x, out=y, workspace=self.ws)
        if name in self.adapters:
            before.copy_(y)
            a, b = self.adapters[name]
            lowbit.lowbit_lora_accumulate(x, self.ids, a, b, y, ranks=self.ranks, scales=self.scales,
                                          workspace=self.ws)

    def step(self):
        import torch

        c, s, n, k = self.embed
        lowbit.lowbit_embed(self.fmt, c, s, n, k, self.last, out=self.emb)
        self.r0.copy_(self.emb)
        lowbit.lowbit_norm_residual(None, self.r0, pre="rms", pre_w=self.w[0], x_out=self.x0)
        self.project("gu", self.x0, self.h, self.h0)
        lowbit.lowbit_silu_mul(self.h, out=self.z)
        self.project("dn", self.z, self.y, self.y0)
        lowbit.lowbit_norm_residual(self.y, self.r0, post="rms", post_w=self.w[1], gate=self.gate, scale=0.5,
                                    pre="layer", pre_w=self.w[2], r_out=self.r1, x_out=self.x1)
        self.project("head", self.x1, self.logits, None)
        rep, freq, pres = self.penalties
        lowbit.lowbit_logits_process(
            self.logits, tokens=self.tokens, prompt_len=self.prompt_len, total_len=self.total_len, repetition=rep,
            frequency=freq, presence=pres, bias_ids=self.bias_ids, bias_vals=self.bias_vals, mask=self.mask,
            mask_row=self.mask_row, out=self.out, idx=self.idx, val=self.val, workspace=self.ws)
        # the token joins its request's
        self.last.copy_(self.idx)
        at = self.total_len.long().unsqueeze(1)
        self.tokens.scatter_(1, at, self.idx.unsqueeze(1))
        self.total_len.add_(1)
        return torch

    def reset(self):
        self.tokens.copy_(self.tokens0)
        self.total_len.copy_(self.prompt_len)
        self.last.copy_(self.last0)


def _np(t):
    return t.cpu().double().numpy()


def _check_stages(m, before):
    """Each stage of the step just run, against 64 bits on the inputs it got."""
    of = oracle.Q1 if m.fmt == "q1" else oracle.T2
    u = {name: oracle.gemv(of, c, s, n, k, host_u16(x)) for name, x in
         (("gu", m.x0), ("dn", m.z), ("head", m.x1)) for c, s, n, k in [m.host[name]]}
    assert_close(_np(m.h0), u["gu"], "gate+up")
    assert_close(_np(m.y0), u["dn"], "down")
    assert_close(_np(m.logits), u["head"], "head")
    for name, x, y0, y in (("gu", m.x0, m.h0, m.h), ("dn", m.z, m.y0, m.y)):
        a, b = m.adapters[name]
        want, bound = plain64.lora(_np(x), _np(m.ids).astype(int), _np(a), _np(b), _np(y0), _np(m.ranks).astype(int),
                                   _np(m.scales))
        assert (np.abs(_np(y) - want) <= bound).all(), name
    w = [_np(t) for t in m.w]
    args = (None, _np(m.r0), None, None, None, None, 1.0, "rms", w[0], None, 1e-6)
    _, x = plain64.norm_residual(*args)
    assert (np.abs(_np(m.x0) - x) <= plain64.norm_residual_bound(*args, "float32", "float16")[1]).all()
    args = (_np(m.y), _np(m.r0), "rms", w[1], None, _np(m.gate), 0.5, "layer", w[2], None, 1e-6)
    r, x = plain64.norm_residual(*args)
    er, ex = plain64.norm_residual_bound(*args, "float32", "float16")
    assert (np.abs(_np(m.r1) - r) <= er).all() and (np.abs(_np(m.x1) - x) <= ex).all()
    host = lambda t: t.cpu().numpy()  # noqa: E731
    out, idx, val, bound = plain64.logits_process(
        _np(m.logits), before[0], host(m.prompt_len), before[1], *[host(t) for t in m.penalties],
        bias_ids=host(m.bias_ids), bias_vals=host(m.bias_vals), mask=host(m.mask), mask_row=host(m.mask_row))
    got, gidx = _np(m.out), host(m.idx)
    fine = np.isfinite(out)
    assert np.array_equal(np.isfinite(got), fine) and (np.abs(got - out)[fine] <= 1.01 * bound[fine]).all()
    for i in range(B):
        assert got[i, gidx[i]] == got[i].max() and _np(m.val)[i] == got[i, gidx[i]]
        top = np.sort(out[i][fine[i]])[-2:]
        if top[1] - top[0] > 4 * bound[i].max():
            assert gidx[i] == idx[i]


@pytest.mark.parametrize("fmt", ["q1", "t2"])
def test_decode_steps_eager_and_as_a_graph(fmt):
    import torch

    say(f"decode steps {fmt}")
    m = Model(fmt, 77)
    eager = []
    for _ in range(8):
        before = (m.tokens.cpu().numpy(), m.total_len.cpu().numpy())
        m.step()
        torch.cuda.synchronize()
        _check_stages(m, before)
        eager.append((m.idx.clone(), m.out.clone(), m.r1.clone()))
    for i in range(B):  # the tokens lie behind the prompts, the rest is as it was
        p, t = int(m.prompt_len[i]), int(m.total_len[i])
        assert t == p + 8 and m.tokens[i, p:t].tolist() == [int(e[0][i]) for e in eager]
        assert torch.equal(m.tokens[i, t:], m.tokens0[i, t:])
    m.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    m.reset()
    for step, (idx, out, r1) in enumerate(eager):
        for t in (m.h, m.y, m.logits, m.out, m.r1, m.x1, m.val):
            t.fill_(7.0)
        m.ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.idx, idx) and torch.equal(m.out, out) and torch.equal(m.r1, r1), step
