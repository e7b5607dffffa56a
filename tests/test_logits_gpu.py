"""lowbit_logits_process against its plain form in 64 bits.

Most inputs are small dyadic numbers (logits and biases in eighths, penalties
powers of two and quarters), for which every FP32 operation is exact: outputs
and indices then have to be equal, ties among them.  Others are held to a
bound that counts each operation's rounding."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64
from tests.helpers import GUARD_BYTE, guarded, guards_intact, say

pytestmark = pytest.mark.gpu


def _dev(a):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _case(b, n, hist, nbias, masked, seed, dyadic=True, mask_rows=None):
    g = np.random.default_rng(seed)
    d = {}
    if dyadic:
        d["y"] = (g.integers(-40, 41, (b, n)) / 8).astype(np.float32)
        d["repetition"] = g.choice([1.0, 2.0, 4.0, 0.5], b).astype(np.float32)
        d["frequency"] = (g.integers(0, 5, b) / 4).astype(np.float32)
        d["presence"] = (g.integers(0, 5, b) / 4).astype(np.float32)
    else:
        d["y"] = (3 * g.standard_normal((b, n))).astype(np.float32)
        d["repetition"] = g.uniform(1, 1.5, b).astype(np.float32)
        d["frequency"] = g.uniform(0, 0.5, b).astype(np.float32)
        d["presence"] = g.uniform(0, 0.5, b).astype(np.float32)
    if hist:
        d["tokens"] = (g.random((b, hist)) ** 3 * n).astype(np.int32)
        d["tokens"][g.random((b, hist)) < 0.05] = -1
        d["tokens"][g.random((b, hist)) < 0.02] = n
        d["total_len"] = g.integers(0, hist + 1, b).astype(np.int32)
        d["prompt_len"] = (d["total_len"] * g.random(b)).astype(np.int32)
        d["total_len"][0] = hist
    if nbias:
        d["bias_ids"] = g.integers(-2, n + 2, (b, nbias)).astype(np.int32)
        d["bias_ids"][:, nbias // 2:] = d["bias_ids"][:, :nbias - nbias // 2]  # listed twice
        d["bias_vals"] = (g.integers(-80, 81, (b, nbias)) / 8).astype(np.float32)
        d["bias_len"] = g.integers(0, nbias + 1, b).astype(np.int32)
        d["bias_len"][0] = nbias
    if masked:
        rows = mask_rows or b
        words = (n + 31) // 32
        d["mask"] = g.integers(-2 ** 31, 2 ** 31, (rows, words)).astype(np.int32)
        if mask_rows:
            d["mask_row"] = g.integers(-1, mask_rows + 1, b).astype(np.int32)
        else:
            d["mask"][b // 2] = 0
    return d


def _run(d, y=None, **over):
    args = {k: _dev(v) for k, v in d.items() if k != "y"}
    args.update(over)
    return lowbit.lowbit_logits_process(_dev(d["y"]) if y is None else y, **args)


def _same(got, want):
    got = got.cpu().double().numpy()
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:5]


SIZES = [(1, 1, 1, 1), (1, 31, 5, 3), (3, 4096, 700, 40), (2, 4097, 1, 0), (5, 8193, 300, 7), (17, 3001, 64, 5),
         (1, 151936, 2000, 64), (9, 32003, 1000, 17)]


@pytest.mark.parametrize("b,n,hist,nbias", SIZES)
@pytest.mark.parametrize("masked", [False, True])
def test_exact_on_dyadic_inputs(b, n, hist, nbias, masked):
    import torch

    say(f"logits b={b} n={n} hist={hist} bias={nbias} mask={masked}")
    d = _case(b, n, hist, nbias, masked, 10 + b + n)
    out = torch.empty((b, n), dtype=torch.float32, device="cuda")
    _, idx, val = _run(d, out=out)
    want, widx, wval, _ = plain64.logits_process(**d)
    _same(out, want)
    _same(idx, widx)
    _same(val, wval)
    # the token alone, and the logits alone
    none, idx2, _ = _run(d)
    assert none is None and torch.equal(idx2, idx)
    out2, a, b_ = _run(d, out=torch.empty_like(out), top1=False)
    assert a is None and b_ is None and torch.equal(out2, out)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_types_and_rounding(dtype):
    import torch

    d = _case(6, 20011, 900, 30, True, 77, dyadic=False)
    y = torch.from_numpy(d["y"]).to(getattr(torch, dtype)).cuda()
    d["y"] = y.cpu().double().numpy()
    out = torch.empty(y.shape, dtype=torch.float32, device="cuda")
    _, idx, val = _run(d, y=y, out=out)
    want, widx, wval, bound = plain64.logits_process(**d)
    got, idx, val = out.cpu().double().numpy(), idx.cpu().numpy(), val.cpu().double().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    assert (np.abs(got - np.where(fine, want, 0))[fine] <= 1.01 * bound[fine]).all()
    for i in range(6):
        if idx[i] >= 0:
            assert got[i, idx[i]] == val[i] == got[i].max() and idx[i] == int(np.argmax(got[i]))
        top = np.sort(want[i])[-2:]
        if np.isneginf(top).all():
            assert idx[i] == -1 == widx[i]
        elif top[1] - top[0] > 4 * bound[i].max():
            assert idx[i] == widx[i]


def test_each_part_alone():
    d = _case(4, 9001, 500, 33, True, 5)
    for keys in (["tokens", "total_len"], ["tokens", "total_len", "prompt_len", "repetition"], ["tokens", "frequency"],
                 ["tokens", "presence", "prompt_len"], ["bias_ids", "bias_vals"], ["bias_ids", "bias_vals", "bias_len"],
                 ["mask"], []):
        say("logits", keys)
        part = {k: d[k] for k in ["y"] + keys}
        import torch

        out = torch.empty((4, 9001), dtype=torch.float32, device="cuda")
        _, idx, val = _run(part, out=out)
        want, widx, wval, _ = plain64.logits_process(**part)
        _same(out, want)
        _same(idx, widx)
        _same(val, wval)


def test_mask_rows_shared_between_requests():
    import torch

    d = _case(12, 5000, 100, 0, True, 6, mask_rows=3)
    assert {-1, 3} <= set(d["mask_row"].tolist())
    out = torch.empty((12, 5000), dtype=torch.float32, device="cuda")
    _, idx, val = _run(d, out=out)
    want, widx, wval, _ = plain64.logits_process(**d)
    _same(out, want)
    _same(idx, widx)
    _same(val, wval)


def test_infinities_nan_and_lengths_out_of_range():
    import torch

    d = _case(6, 5003, 40, 6, True, 8)
    y = d["y"]
    y[0, 17] = np.nan       # allowed or not, as the mask has it
    y[1, :] = -np.inf       # nothing but -inf: the lowest allowed one
    y[2, 100] = np.inf
    y[4, 3] = np.float32(-3.4e38)  # the type's lowest value
    d["total_len"][2] = 10 ** 6
    d["total_len"][4] = -5
    d["prompt_len"][5] = 10 ** 6
    d["bias_len"][1] = -1
    d["bias_len"][2] = 1000
    d["mask"][0, 17 // 32] |= 1 << 17
    out = torch.empty((6, 5003), dtype=torch.float32, device="cuda")
    for hidden in (False, True):
        if hidden:  # a NaN in a masked place is seen by nobody
            d["mask"][0, 17 // 32] &= ~np.int32(1 << 17)
        _, idx, val = _run(d, out=out)
        want, widx, wval, bound = plain64.logits_process(**d)
        got = out.cpu().double().numpy()
        want32 = want.astype(np.float32).astype(np.float64)
        assert np.array_equal(got, want32, equal_nan=True)
        _same(idx, widx)
        _same(val, wval.astype(np.float32).astype(np.float64))
        assert np.isnan(got[0, 17]) != hidden


def test_one_token_many_times_and_repeated_biases():
    import torch

    n, hist = 4200, 33000
    d = dict(y=np.zeros((2, n), np.float32), tokens=np.full((2, hist), 4100, np.int32),
             prompt_len=np.array([0, 32999], np.int32), frequency=np.array([0.5, 0.5], np.float32),
             presence=np.array([0.25, 0.25], np.float32), repetition=np.array([2.0, 2.0], np.float32))
    # 1e8 + 1 - 1e8: only the list's order gives these bits
    vals = np.tile(np.array([1e8, 1.0, -1e8, 3.0], np.float32), 70)
    d["bias_ids"] = np.full((2, 280), 7, np.int32)
    d["bias_vals"] = np.stack([vals, vals[::-1]])
    out = torch.empty((2, n), dtype=torch.float32, device="cuda")
    _run(d, out=out)
    got = out.cpu().numpy()
    assert got[0, 4100] == np.float32(-16500.25) and got[1, 4100] == np.float32(-0.75)
    for i in range(2):
        s = np.float32(0)
        for v in d["bias_vals"][i]:
            s = np.float32(s + v)
        assert got[i, 7] == s


def test_strides_in_place_and_guards():
    import torch

    d = _case(5, 3001, 64, 9, True, 21)
    want, widx, wval, _ = plain64.logits_process(**d)
    wide = torch.full((5, 3300), 7.0, device="cuda")
    y = wide[:, 11:11 + 3001]
    y.copy_(_dev(d["y"]))
    tok = torch.full((5, 80), 3, dtype=torch.int32, device="cuda")
    tok[:, 5:69] = _dev(d["tokens"])
    mask = torch.full((5, 100), -1, dtype=torch.int32, device="cuda")
    mask[:, 3:3 + 94] = _dev(d["mask"])
    got, idx, val = _run(d, y=y, tokens=tok[:, 5:69], mask=mask[:, 3:97], out=y)
    assert got is y
    _same(y, want)
    _same(idx, widx)
    assert bool((wide[:, :11] == 7.0).all()) and bool((wide[:, 3012:] == 7.0).all())
    raw, out = guarded((7, 3001), torch.float32)
    iraw, idx = guarded((7,), torch.int32)
    vraw, val = guarded((7,), torch.float32)
    need = lowbit.lowbit_logits_workspace_bytes(3001, 5)
    wraw, ws = guarded((need,), torch.uint8)
    _run(d, out=out[:5], idx=idx, val=val, workspace=ws)
    torch.cuda.synchronize()
    _same(out[:5], want)
    _same(idx[:5], widx)
    for r in (raw, iraw, vraw, wraw):
        assert guards_intact(r)
    for t in (out[5:], idx[5:], val[5:]):
        assert bool((t.contiguous().view(torch.uint8) == GUARD_BYTE).all())


def test_graph_replays_with_growing_lengths():
    import torch

    d = _case(4, 20000, 300, 20, True, 31)
    t = {k: _dev(v) for k, v in d.items()}
    out = torch.empty((4, 20000), dtype=torch.float32, device="cuda")
    idx, val = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    ws = torch.empty(lowbit.lowbit_logits_workspace_bytes(20000, 4), dtype=torch.uint8, device="cuda")
    rest = {k: v for k, v in t.items() if k != "y"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lowbit.lowbit_logits_process(t["y"], out=out, idx=idx, val=val, workspace=ws, **rest)
    for step in range(4):
        d["total_len"] = np.minimum(d["total_len"] + step, 300).astype(np.int32)
        t["total_len"].copy_(torch.from_numpy(d["total_len"]))
        out.fill_(3.0)
        ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        want, widx, wval, _ = plain64.logits_process(**d)
        _same(out, want)
        _same(idx, widx)
        _same(val, wval)


def test_offsets_past_32_bits():
    import torch

    n, ld = 5003, (1 << 28) + 3  # 20 rows: 5.4e9 logits, 21 GB
    d = _case(20, n, 64, 5, True, 41)
    want, widx, wval, _ = plain64.logits_process(**d)
    wide = torch.empty(20, ld, device="cuda")
    y = wide[:, 77:77 + n]
    y.copy_(_dev(d["y"]))
    _, idx, val = _run(d, y=y, out=y)
    _same(y, want)
    _same(idx, widx)
    _same(val, wval)


@pytest.mark.parametrize("b", [3, 40])
def test_more_biases_than_threads_and_than_lds_holds(b):
    """Long lists of biases: later entries are not kept by a thread, and past
    256 in one part the list itself is searched."""
    import torch

    n = 20000
    for nbias, top in ((1500, n), (700, 900), (3000, 3000)):
        g = np.random.default_rng(nbias)
        d = _case(b, n, 50, nbias, True, nbias)
        d["bias_ids"] = g.integers(0, top, (b, nbias)).astype(np.int32)
        d["bias_len"][:] = nbias
        out = torch.empty((b, n), dtype=torch.float32, device="cuda")
        _, idx, val = _run(d, out=out)
        want, widx, wval, _ = plain64.logits_process(**d)
        _same(out, want)
        _same(idx, widx)
        _same(val, wval)


@pytest.mark.parametrize("b,n", [(64, 151936), (400, 20001), (70, 60000)])
def test_long_lists_of_tokens(b, n):
    """The large parts: lists of 16384 tokens and more."""
    import torch

    g = np.random.default_rng(b)
    hist = 16500
    d = dict(y=(g.integers(-40, 41, (b, n)) / 8).astype(np.float32),
             tokens=(g.random((b, hist)) ** 4 * n).astype(np.int32),
             total_len=g.integers(0, hist + 1, b).astype(np.int32), repetition=np.full(b, 2.0, np.float32),
             frequency=np.full(b, 0.25, np.float32), presence=np.full(b, 0.5, np.float32))
    d["prompt_len"] = (d["total_len"] // 2).astype(np.int32)
    rows = g.choice(b, 4, replace=False)
    out = torch.empty((b, n), dtype=torch.float32, device="cuda")
    _, idx, val = _run(d, out=out)
    want, widx, wval, _ = plain64.logits_process(**{k: v[rows] for k, v in d.items()})
    _same(out[rows], want)
    _same(idx[rows], widx)
    _same(val[rows], wval)
    assert torch.equal(idx.long(), out.max(dim=1).indices) or torch.equal(out.max(dim=1).values, val)


# (b, n, tokens, biases): parts of 4096, 8192, 19456, 2048 and 2048 tokens; in batches of 8 of 1024 or 2048
@pytest.mark.parametrize("b,n,hist,nbias", [(64, 32000, 2048, 1500), (64, 50001, 300, 700), (64, 120001, 16400, 1100),
                                            (24, 32003, 700, 600), (47, 32000, 500, 300)])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_every_part_size_with_everything(b, n, hist, nbias, dtype):
    """More biases than threads, and than LDS holds for one part, shared mask
    rows, each type, in place where that can be: sampled rows against the plain
    form, all rows against themselves in small batches, every token against its
    row."""
    import torch

    say(f"logits b={b} n={n} hist={hist} bias={nbias} {dtype}")
    d = _case(b, n, hist, nbias, True, b + n, mask_rows=5)
    g = np.random.default_rng(n)
    crowd = g.random((b, nbias)) < 0.5
    d["bias_ids"][crowd] = g.integers(0, 700, crowd.sum())
    y = torch.from_numpy(d["y"]).to(getattr(torch, dtype)).cuda()
    t = {k: _dev(v) for k, v in d.items() if k != "y"}
    parts = []
    for i in range(0, b, 8):
        rows = {k: v if k == "mask" else v[i:i + 8] for k, v in t.items()}
        out = torch.empty(y[i:i + 8].shape, dtype=torch.float32, device="cuda")
        parts.append(lowbit.lowbit_logits_process(y[i:i + 8], out=out, **rows))
    out = y if dtype == "float32" else torch.empty((b, n), dtype=torch.float32, device="cuda")
    out, idx, val = lowbit.lowbit_logits_process(y, out=out, **t)
    for at, got in enumerate((out, idx, val)):
        assert torch.equal(got, torch.cat([p[at] for p in parts])), at
    # the lowest of a row's largest; -1 where nothing is allowed
    first = torch.where(out == val[:, None], torch.arange(n, device="cuda"), n).amin(dim=1)
    none = torch.isneginf(val)
    assert torch.equal(val, out.amax(dim=1)) and torch.equal(idx.long(), torch.where(none, -1, first))
    rows = np.unique(np.concatenate([[0, b - 1], g.choice(b, 3, replace=False)]))
    want, widx, wval, _ = plain64.logits_process(**{k: v if k == "mask" else v[rows] for k, v in d.items()})
    _same(out[rows], want)
    _same(idx[rows], widx)
    _same(val[rows], wval)


@pytest.mark.parametrize("b,n", [(64, 151936), (400, 20001), (70, 60000)])
def test_tokens_of_every_row_with_long_lists(b, n):
    """The lowest of a row's largest, in rows full of ties."""
    import torch

    g = np.random.default_rng(b + 1)
    hist = 16500
    y = torch.from_numpy((g.integers(-40, 41, (b, n)) / 8).astype(np.float32)).cuda()
    out = torch.empty_like(y)
    _, idx, val = lowbit.lowbit_logits_process(
        y, tokens=_dev((g.random((b, hist)) ** 4 * n).astype(np.int32)),
        total_len=_dev(g.integers(0, hist + 1, b).astype(np.int32)), repetition=_dev(np.full(b, 2.0, np.float32)), out=out)
    assert torch.equal(val, out.amax(dim=1))
    first = torch.where(out == val[:, None], torch.arange(n, device="cuda"), n).amin(dim=1)
    assert torch.equal(idx.long(), first)


@pytest.mark.parametrize("same", [False, True])
def test_the_longest_list_of_biases_in_one_part(same):
    """16384 entries that fall together, every id once or one id for all."""
    import torch

    n, nbias = 32000, 16384
    g = np.random.default_rng(3)
    d = _case(3, n, 50, 0, False, 3)
    d["bias_ids"] = np.stack([np.full(nbias, 77) if same else g.permutation(nbias) % 1000 for _ in range(3)]).astype(np.int32)
    d["bias_vals"] = (g.integers(-8, 9, (3, nbias)) / 8).astype(np.float32)
    out = torch.empty((3, n), dtype=torch.float32, device="cuda")
    _, idx, val = _run(d, out=out)
    want, widx, wval, _ = plain64.logits_process(**d)
    _same(out, want)
    _same(idx, widx)
    _same(val, wval)


@pytest.mark.parametrize("b,n,top", [(64, 151936, 151936), (8, 151936, 151936), (64, 32000, 1000), (3, 32000, 1)])
def test_long_lists_of_biases_are_bounded_work(b, n, top):
    """16384 biases a row: a walk over the list for each group of tokens, not
    for each token (that was 127 ms for the first of these calls)."""
    import torch

    nbias = 16384
    ids = torch.stack([torch.randperm(top, device="cuda").repeat((nbias + top - 1) // top)[:nbias] for _ in range(b)]).int()
    y = torch.randn(b, n, device="cuda")
    args = dict(bias_ids=ids, bias_vals=torch.randn(b, nbias, device="cuda"), out=torch.empty_like(y))
    lowbit.lowbit_logits_process(y, **args)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out, _, _ = lowbit.lowbit_logits_process(y, **args)
    end.record()
    end.synchronize()
    want = y[0].double().index_add(0, ids[0].long(), args["bias_vals"][0].double())
    # at most 16384 additions of values below 6
    assert bool(((out[0].double() - want).abs() <= nbias * 2.0 ** -24 * 6 * (nbias / min(top, nbias))).all())
    assert start.elapsed_time(end) < 20
