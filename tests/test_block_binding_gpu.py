"""What the binding of rope, the 4-bit cache, attention and the draw refuses before the
library is called; other streams, two calls at once, graphs that share a workspace."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests.helpers import say

pytestmark = pytest.mark.gpu

HEADS, D, PAGE = 2, 64, 16


def _f(*shape, dtype="float32"):
    import torch

    return torch.zeros(shape, dtype=getattr(torch, dtype), device="cuda")


def _pages(n=4):
    return _f(n, lowbit.lowbit_kv_page_bytes(HEADS, D, PAGE), dtype="uint8")


def _rope(**over):
    args = dict(x=_f(3, 4, D), positions=_f(3, dtype="int32"), turns=_f(16, dtype="int64"))
    args.update(over)
    return lowbit.lowbit_rope(**args)


def _store(**over):
    args = dict(k=_f(3, HEADS, D), v=_f(3, HEADS, D), slots=_f(3, dtype="int32"), pages=_pages(), page=PAGE,
                positions=_f(3, dtype="int32"), turns=_f(32, dtype="int64"), q=_f(3, 4, D))
    args.update(over)
    return lowbit.lowbit_kv_store(**args)


def _load(**over):
    args = dict(pages=_pages(), page=PAGE, slots=_f(3, dtype="int32"), heads=HEADS, d=D)
    args.update(over)
    return lowbit.lowbit_kv_load(**args)


def _attention(**over):
    args = dict(q=_f(3, 4, D, dtype="float16"), pages=_pages(), page=PAGE, table=_f(3, 2, dtype="int32"),
                lengths=_f(3, dtype="int32"))
    args.update(over)
    return lowbit.lowbit_attention(**args)


def _sample(**over):
    args = dict(y=_f(3, 1000), u=_f(3), temperature=_f(3), top_k=_f(3, dtype="int32"), top_p=_f(3), min_p=_f(3))
    args.update(over)
    return lowbit.lowbit_sample(**args)


CALLS = [_rope, _store, _load, _attention, _sample]


def test_the_plain_calls_pass():
    import torch

    for call in CALLS:
        call()
    torch.cuda.synchronize()


BAD = (TypeError, ValueError, lowbit.LowbitError)


@pytest.mark.parametrize("call,over", [
    (_rope, lambda: dict(x=_f(3, 4, D, dtype="int32"))),
    (_rope, lambda: dict(x=_f(3, 4 * D))),
    (_rope, lambda: dict(x=_f(3, 4, D).cpu())),
    (_rope, lambda: dict(x=_f(3, 4, 2 * D)[..., ::2])),
    (_rope, lambda: dict(positions=_f(2, dtype="int32"))),
    (_rope, lambda: dict(positions=_f(3, dtype="int64"))),
    (_rope, lambda: dict(positions=_f(6, dtype="int32")[::2])),
    (_rope, lambda: dict(turns=_f(33, dtype="int64"))),
    (_rope, lambda: dict(turns=_f(16, dtype="int32"))),
    (_rope, lambda: dict(turns=_f(16))),
    (_rope, lambda: dict(out=_f(3, 4, D - 1))),
    (_rope, lambda: dict(out=_f(2, 4, D))),
    (_rope, lambda: dict(out_dtype="float32")),
    (_rope, lambda: dict(x=_f(1, 4, D).expand(3, 4, D), out=_f(1, 4, D).expand(3, 4, D))),
    (_store, lambda: dict(k=_f(3, HEADS + 1, D))),
    (_store, lambda: dict(v=_f(2, HEADS, D))),
    (_store, lambda: dict(v=_f(3, HEADS, D, dtype="float16"))),
    (_store, lambda: dict(slots=_f(2, dtype="int32"))),
    (_store, lambda: dict(slots=_f(3, dtype="int64"))),
    (_store, lambda: dict(pages=_f(4, 100, dtype="uint8"))),
    (_store, lambda: dict(pages=_pages().float())),
    (_store, lambda: dict(pages=_pages(8)[::2])),
    (_store, lambda: dict(page=24)),
    (_store, lambda: dict(page=32)),
    (_store, lambda: dict(positions=None)),
    (_store, lambda: dict(turns=None, q=None)),
    (_store, lambda: dict(q=_f(2, 4, D))),
    (_store, lambda: dict(q=_f(3, 4, 2 * D))),
    (_store, lambda: dict(q=None, q_out=_f(3, 4, D))),
    (_store, lambda: dict(k=_f(3, HEADS, 96), v=_f(3, HEADS, 96))),
    (_load, lambda: dict(pages=_f(4, 100, dtype="uint8"))),
    (_load, lambda: dict(page=8)),
    (_load, lambda: dict(slots=_f(3))),
    (_load, lambda: dict(heads=HEADS + 1)),
    (_load, lambda: dict(d=96)),
    (_load, lambda: dict(k_out=_f(3, HEADS, D, dtype="int32"))),
    (_load, lambda: dict(k_out=_f(2, HEADS, D))),
    (_load, lambda: dict(k_out=_f(3, HEADS, D), v_out=_f(3, HEADS, D, dtype="float16"))),
    (_attention, lambda: dict(q=_f(3, 4, D))),
    (_attention, lambda: dict(q=_f(3, 4 * D, dtype="float16"))),
    (_attention, lambda: dict(pages=_f(4, 100, dtype="uint8"))),
    (_attention, lambda: dict(page=48)),
    (_attention, lambda: dict(table=_f(3, 2, dtype="int64"))),
    (_attention, lambda: dict(table=_f(6, dtype="int32"))),
    (_attention, lambda: dict(table=_f(3, 4, dtype="int32")[:, ::2])),
    (_attention, lambda: dict(lengths=_f(2, dtype="int32"))),
    (_attention, lambda: dict(lengths=_f(3))),
    (_attention, lambda: dict(q=_f(4, 4, D, dtype="float16"))),
    (_attention, lambda: dict(q_start=_f(3, dtype="int32"))),
    (_attention, lambda: dict(q_start=_f(4, dtype="int64"))),
    (_attention, lambda: dict(q_start=_f(4, dtype="int32"), max_q=0)),
    (_attention, lambda: dict(max_q=-1)),
    (_attention, lambda: dict(scale=float("nan"))),
    (_attention, lambda: dict(scale=float("inf"))),
    (_attention, lambda: dict(out=_f(3, 4, D + 1, dtype="float16"))),
    (_attention, lambda: dict(out=_f(3, 4, D, dtype="int32"))),
    (_attention, lambda: dict(lse=_f(3, 3))),
    (_attention, lambda: dict(lse=_f(3, 4, dtype="float16"))),
    (_attention, lambda: dict(workspace=_f(8, dtype="uint8"))),
    (_sample, lambda: dict(y=_f(3, 1000, dtype="int32"))),
    (_sample, lambda: dict(y=_f(1000, 3).t())),
    (_sample, lambda: dict(u=_f(2))),
    (_sample, lambda: dict(u=_f(3, dtype="float16"))),
    (_sample, lambda: dict(temperature=_f(2))),
    (_sample, lambda: dict(top_k=_f(3))),
    (_sample, lambda: dict(top_p=_f(3, dtype="float64"))),
    (_sample, lambda: dict(min_p=_f(6)[::2])),
    (_sample, lambda: dict(idx=_f(3, dtype="int64"))),
    (_sample, lambda: dict(idx=_f(2, dtype="int32"))),
    (_sample, lambda: dict(prob=_f(2))),
    (_sample, lambda: dict(workspace=_f(8, dtype="uint8"))),
])
def test_refusals(call, over):
    with pytest.raises(BAD):
        call(**over())


class _OtherDevice:
    device_index = 1
    cuda_stream = 0


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device_is_refused(call):
    with pytest.raises(ValueError):
        call(stream=_OtherDevice())


def _state(seed, b=3, ctx=700):
    """Arguments for attention and a draw, and their results on the current stream."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    n = b * (ctx // PAGE + 1)
    pages = _pages(n)
    slots = torch.arange(n * PAGE, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n * PAGE, HEADS, D, generator=g, device="cuda") for _ in range(2))
    lowbit.lowbit_kv_store(k, v, slots, pages, PAGE)
    att = dict(q=torch.randn(b, 8, D, generator=g, device="cuda").half(), pages=pages, page=PAGE,
               table=torch.randperm(n, generator=g, device="cuda").int().view(b, -1),
               lengths=torch.randint(1, ctx, (b,), generator=g, device="cuda").int())
    draw = dict(y=torch.randn(b, 70001, generator=g, device="cuda") * 3, u=torch.rand(b, generator=g, device="cuda"),
                top_k=torch.tensor([0, 50, 3000], dtype=torch.int32, device="cuda"),
                top_p=torch.tensor([0.9, 0.8, 1.0], device="cuda"))
    return att, draw, lowbit.lowbit_attention(**att), lowbit.lowbit_sample(**draw)[0]


def test_two_streams_at_once():
    import torch

    say("two streams")
    states = [_state(s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (att, draw, _, _) in enumerate(states):
            got[i].append((lowbit.lowbit_attention(**att, stream=streams[i]),
                           lowbit.lowbit_sample(**draw, stream=streams[i])[0]))
    torch.cuda.synchronize()
    for i, (_, _, out, idx) in enumerate(states):
        assert all(torch.equal(a, out) and torch.equal(b, idx) for a, b in got[i])


def test_two_graphs_share_a_workspace_and_read_new_inputs():
    """Replayed in turn on one stream, with other inputs, lengths and settings than at
    their capture, and eager calls between them."""
    import torch

    say("two graphs, one workspace")
    b = 3
    ws = _f(max(lowbit.lowbit_attention_workspace_bytes(b, b, 8, HEADS, D),
                lowbit.lowbit_sample_workspace_bytes(70001, b)), dtype="uint8")
    states = [_state(s) for s in (3, 4)]
    held, outs, graphs = [], [], []
    for att, draw, _, _ in states:
        a = {k: v.clone() if hasattr(v, "clone") else v for k, v in att.items()}
        d = {k: v.clone() for k, v in draw.items()}
        out, idx, prob = torch.empty_like(a["q"]), _f(b, dtype="int32"), _f(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lowbit.lowbit_attention(**a, out=out, workspace=ws)
            lowbit.lowbit_sample(**d, idx=idx, prob=prob, workspace=ws)
        held.append((a, d))
        outs.append((out, idx))
        graphs.append(graph)
    for turn in range(6):
        ws.fill_(0xFF if turn % 2 else 0)
        for i, graph in enumerate(graphs):
            att, draw, out, idx = states[(i + turn) % 2]
            for mine, given in zip(held[i], (att, draw)):
                for key, value in given.items():
                    if hasattr(value, "clone"):
                        mine[key].copy_(value)
            graph.replay()
            assert torch.equal(lowbit.lowbit_attention(**att), out)
            torch.cuda.synchronize()
            assert torch.equal(outs[i][0], out) and torch.equal(outs[i][1], idx), (turn, i)


@pytest.mark.parametrize("op", ["rope", "load", "attention", "sample"])
def test_outputs_on_another_stream_do_not_reuse_its_memory(op):
    """What the current stream freed may still be written by work that waits there: a call
    on another stream gets other memory for its outputs."""
    import torch

    side = torch.cuda.Stream()
    x, pos, turns = _f(4000, 64, D), _f(4000, dtype="int32"), _f(32, dtype="int64")
    q, table, length = _f(4000, 64, D, dtype="float16"), _f(4000, 1, dtype="int32"), _f(4000, dtype="int32") + 1
    y, u, pages = _f(200000, 8), _f(200000), _pages(8)
    torch.cuda.synchronize()

    def run():
        if op == "rope":
            return [lowbit.lowbit_rope(x, pos, turns, stream=side)]
        if op == "load":
            return list(lowbit.lowbit_kv_load(pages, PAGE, _f(30000, dtype="int32"), HEADS, D, stream=side))
        if op == "attention":
            return [lowbit.lowbit_attention(q, pages, PAGE, table, length, stream=side)]
        return [lowbit.lowbit_sample(y[:60000], u[:60000], stream=side)[0]]

    sizes = [(t.numel(), t.dtype) for t in run()]
    torch.cuda.synchronize()
    freed = [torch.empty(n, dtype=t, device="cuda") for n, t in sizes]
    kept = {t.data_ptr() for t in freed}
    del freed
    outs = run()
    torch.cuda.synchronize()
    assert not kept & {t.data_ptr() for t in outs}


@pytest.mark.parametrize("call,over", [
    (_rope, lambda: dict(x=_f(0, 4, D), positions=_f(0, dtype="int32"))),
    (_store, lambda: dict(k=_f(0, HEADS, D), v=_f(0, HEADS, D), slots=_f(0, dtype="int32"), q=None)),
    (_store, lambda: dict(pages=_pages(0))),
    (_load, lambda: dict(slots=_f(0, dtype="int32"))),
    (_load, lambda: dict(pages=_pages(0))),
    (_attention, lambda: dict(q=_f(0, 4, D, dtype="float16"), table=_f(0, 2, dtype="int32"),
                              lengths=_f(0, dtype="int32"))),
    (_attention, lambda: dict(table=_f(3, 0, dtype="int32"))),
    (_attention, lambda: dict(pages=_pages(0))),
    (_sample, lambda: dict(y=_f(0, 1000), u=_f(0))),
    (_sample, lambda: dict(y=_f(3, 0))),
])
def test_nothing_to_do_is_refused(call, over):
    with pytest.raises(BAD):
        call(**over())


def test_the_same_slot_twice_stays_inside():
    """Two tokens of one call for one slot: one of them or a mixture of both is held there (which
    is not said), and nothing beside it is touched."""
    import torch

    say("slots twice")
    g = torch.Generator(device="cuda").manual_seed(5)
    for m in (2, 9, 500):
        pages = _pages(8)
        lowbit.lowbit_kv_store(torch.randn(128, HEADS, D, generator=g, device="cuda"),
                               torch.randn(128, HEADS, D, generator=g, device="cuda"),
                               torch.arange(128, dtype=torch.int32, device="cuda"), pages, PAGE)
        k0, v0 = lowbit.lowbit_kv_load(pages, PAGE, torch.arange(128, dtype=torch.int32, device="cuda"), HEADS, D)
        lowbit.lowbit_kv_store(torch.randn(m, HEADS, D, generator=g, device="cuda"),
                               torch.randn(m, HEADS, D, generator=g, device="cuda"),
                               _f(m, dtype="int32") + 37, pages, PAGE)
        k, v = lowbit.lowbit_kv_load(pages, PAGE, torch.arange(128, dtype=torch.int32, device="cuda"), HEADS, D)
        others = np.r_[0:37, 38:128]
        assert torch.equal(k[others], k0[others]) and torch.equal(v[others], v0[others])
        assert torch.isfinite(k[37]).all() and torch.isfinite(v[37]).all()
