"""lowbit_lora_accumulate against its plain form in 64 bits: one row to more
than a plan's chunk, shared and absent adapters, ranks from 0, every type
pair, strided y, and the values at which FP16 pairs could go wrong."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64
from tests.helpers import GUARD_BYTE, guarded, guards_intact, say

pytestmark = pytest.mark.gpu

NAMES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def _t(a, name):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, NAMES[name])).cuda()


def _case(m, k, n, r, slots, xt, yt, ids=None, ragged=False, seed=1, scaled=True):
    import torch

    g = np.random.default_rng(seed)
    d = dict(x=_t(g.standard_normal((m, k)), xt), a=_t(g.standard_normal((slots, r, k)) / k ** 0.5, xt),
             b=_t(g.standard_normal((slots, n, r)) * 0.3, xt), y=_t(g.standard_normal((m, n)), yt))
    if ids is None:
        ids = g.integers(-1, slots + 1, m)
    d["ids"] = torch.from_numpy(np.asarray(ids, dtype=np.int32)).cuda()
    if ragged:
        ranks = g.integers(0, r + 1, slots)
        ranks[0] = 0
        ranks[-1] = r
        d["ranks"] = torch.from_numpy(ranks.astype(np.int32)).cuda()
    if scaled:
        d["scales"] = torch.from_numpy(g.uniform(0.5, 2.0, slots).astype(np.float32)).cuda()
    return d


def _want(d, y, yt):
    v = {k: t.cpu().double().numpy() for k, t in d.items() if k != "y"}
    return plain64.lora(v["x"], v["ids"], v["a"], v["b"], y, v.get("ranks"), v.get("scales"), NAMES[yt])


def _check(got, want, bound):
    got = got.cpu().double().numpy()
    off = np.abs(got - want) - bound
    assert np.isfinite(got).all() and off.max() <= 0, \
        f"off by {np.abs(got - want).max():.3g}, over the bound by {off.max():.3g} at {np.argwhere(off > 0)[:4].tolist()}"


SHAPES = [(1, 128, 1, 8, 1), (1, 2048, 6144, 16, 8), (8, 1280, 700, 64, 16), (3, 8, 17, 8, 2), (16, 5120, 130, 24, 3),
          (17, 136, 1000, 40, 5), (64, 384, 515, 128, 70), (65, 640, 333, 16, 4), (200, 2176, 257, 40, 24),
          (7, 17408, 64, 256, 2), (300, 256, 1025, 32, 300), (1030, 128, 96, 8, 3),
          # one launch with 32 and 64 ranks; several items of one adapter; more rows than a plan keeps in registers
          (9, 512, 300, 32, 4), (12, 256, 700, 64, 5), (16, 640, 129, 48, 16), (40, 384, 300, 128, 3),
          (64, 256, 100, 16, 1), (5000, 64, 40, 8, 2), (9000, 8, 16, 8, 700),
          # items of 32 rows with the most ranks; ranks that end inside a 32 at outputs that end inside a wave's
          (150, 264, 530, 256, 3), (100, 128, 515, 200, 2), (130, 128, 2049, 72, 2),
          # as many adapters as there can be
          (40, 8, 16, 8, 4096), (100, 16, 24, 16, 4096), (5000, 8, 16, 8, 4096)]


@pytest.mark.parametrize("m,k,n,r,slots", SHAPES)
@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_matches_plain_form(m, k, n, r, slots, xt, yt):
    import torch

    say(f"lora m={m} k={k} n={n} r={r} slots={slots} {xt} {yt}")
    ragged = (m + r) % 2 == 1
    ids = [slots - 1] if m == 1 else None
    d = _case(m, k, n, r, slots, xt, yt, ids=ids, ragged=ragged, seed=m + k)
    y0 = d["y"].clone()
    got = lowbit.lowbit_lora_accumulate(**d)
    torch.cuda.synchronize()
    assert got is d["y"]
    _check(got, *_want(d, y0.cpu().double().numpy(), yt))
    # equal inputs, equal bits
    again = lowbit.lowbit_lora_accumulate(**{**d, "y": y0})
    assert torch.equal(again, got)


@pytest.mark.parametrize("m", [5, 64, 130, 1000])
def test_row_orders(m):
    """One adapter for all, none for any, long segments, every row its own:
    whichever way rows are grouped, each gets its own sum."""
    import torch

    g = np.random.default_rng(m)
    orders = [np.zeros(m), np.full(m, -1), np.full(m, 9), np.arange(m) % 9, np.sort(g.integers(0, 9, m)),
              np.where(np.arange(m) % 7 == 3, 4, -1), np.arange(m)[::-1] // max(1, m // 9)]
    base = _case(m, 256, 200, 16, 9, "f16", "f32", ids=np.zeros(m), seed=m)
    for ids in orders:
        d = dict(base, ids=torch.from_numpy(ids.astype(np.int32)).cuda(), y=base["y"].clone())
        got = lowbit.lowbit_lora_accumulate(**d)
        _check(got, *_want(d, base["y"].cpu().double().numpy(), "f32"))
        none = torch.from_numpy((ids < 0) | (ids > 8)).cuda()
        assert torch.equal(got[none], base["y"][none])


@pytest.mark.parametrize("off,pad", [(0, 0), (64, 0), (4, 12), (1, 6), (7, 3)])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("m", [4, 90])
def test_slice_of_a_fused_output(off, pad, yt, m):
    import torch

    n = 300
    d = _case(m, 384, n, 16, 3, "bf16", yt, seed=off + pad)
    y0 = d["y"].cpu().double().numpy()
    wide = torch.full((m + 1, off + n + pad), 5.0, dtype=d["y"].dtype, device="cuda")
    wide[:m, off:off + n] = d["y"]
    xw = torch.full((m, 384 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:, 8:392] = d["x"]
    d["y"] = wide[:m, off:off + n]
    got = lowbit.lowbit_lora_accumulate(**{**d, "x": xw[:, 8:392]})
    _check(got, *_want(d, y0, yt))
    assert bool((wide[:m, :off] == 5.0).all()) and bool((wide[:m, off + n:] == 5.0).all())
    assert bool((wide[m] == 5.0).all())


def test_unused_entries_are_not_read():
    """NaN in adapters no row uses, past a slot's rank, and in rows without an
    adapter reach nothing."""
    import torch

    for m in (6, 100):
        d = _case(m, 640, 130, 24, 4, "f16", "f32", ids=np.arange(m) % 3, seed=4)
        d["ids"][4] = -1
        d["ranks"] = torch.tensor([24, 9, 1, 24], dtype=torch.int32, device="cuda")
        y0 = d["y"].clone()
        want = _want(d, y0.cpu().double().numpy(), "f32")
        for s, rank in enumerate([24, 9, 1, 0]):
            d["a"][s, rank:] = float("nan")
            d["b"][s, :, rank:] = float("nan")
        d["x"][4] = float("nan")
        got = lowbit.lowbit_lora_accumulate(**d)
        _check(got, *want)
        # and one in a row's x stays in that row
        d["x"][0, 3] = float("nan")
        got = lowbit.lowbit_lora_accumulate(**{**d, "y": y0})
        assert torch.isnan(got[0]).all() and torch.isfinite(got[1:]).all()


@pytest.mark.parametrize("m", [2, 80])
def test_wide_range_of_the_inner_values(m):
    """v beyond FP16's range, tiny v, and both in one row."""
    import torch

    g = np.random.default_rng(9)
    k, n, r = 512, 96, 16
    d = _case(m, k, n, r, 2, "f16", "f32", ids=np.arange(m) % 2, seed=9, scaled=False)
    a = g.standard_normal((2, r, k)).astype(np.float32)
    a[0, :8] *= 2000.0      # v up to 1e6 and more
    a[1] *= 2.0 ** -20      # FP16 subnormals
    d["a"] = _t(a, "f16")
    d["x"] = _t(g.standard_normal((m, k)) * 30, "f16")
    d["scales"] = torch.tensor([16.0, 2.0 ** -30], device="cuda")
    y0 = torch.zeros(m, n, device="cuda")
    got = lowbit.lowbit_lora_accumulate(**{**d, "y": y0.clone()})
    _check(got, *_want(d, y0.cpu().double().numpy(), "f32"))


def test_infinite_inner_values_follow_the_formula():
    import torch

    d = _case(3, 128, 40, 8, 1, "bf16", "f32", ids=[0, 0, 0], seed=2)
    d["x"][1, 0] = float("inf")
    d["a"][0, :, 0] = 1.0
    d["b"][0] = d["b"][0].abs() + 0.5
    got = lowbit.lowbit_lora_accumulate(**d)
    assert torch.isinf(got[1]).all() and (got[1] > 0).all() and torch.isfinite(got[[0, 2]]).all()


@pytest.mark.parametrize("m", [3, 100])
def test_guards_graph_and_stream(m):
    import torch

    d = _case(m, 1280, 515, 40, 6, "f16", "f32", ragged=True, seed=20)
    y0 = d["y"].clone()
    want = _want(d, y0.cpu().double().numpy(), "f32")
    yraw, y = guarded((m + 1, 515), torch.float32)
    y[:m] = y0
    need = lowbit.lowbit_lora_workspace_bytes(m, 515, 1280, 40, 6)
    wraw, ws = guarded((need,), torch.uint8)
    args = dict(d, y=y[:m], workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lowbit.lowbit_lora_accumulate(**args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(y[:m], *want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lowbit.lowbit_lora_accumulate(**args)
    for rep in range(3):
        y[:m] = y0
        ws.fill_(0x7F)  # stale contents: NaN patterns
        graph.replay()
        torch.cuda.synchronize()
        _check(y[:m], *want)
    assert guards_intact(yraw) and guards_intact(wraw)
    assert bool((y[m].view(torch.uint8) == GUARD_BYTE).all())
    # other rows under the same graph: ids are read when it runs
    d["ids"].copy_(torch.roll(d["ids"], 1))
    y[:m] = y0
    graph.replay()
    _check(y[:m], *_want(d, y0.cpu().double().numpy(), "f32"))


def test_offsets_past_32_bits():
    import torch

    m, k, n, ld = 70, 128, 300, (1 << 26) + 64  # 70 rows: 4.7e9 elements, 9.4 GB
    d = _case(m, k, n, 16, 3, "bf16", "bf16", seed=40)
    y0 = d["y"].cpu().double().numpy()
    want = _want(d, y0, "bf16")
    wide = torch.empty(m, ld, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:5 + n] = d["y"]
    wide[:, ld - 200:ld - 72] = d["x"]
    d["y"], d["x"] = wide[:, 5:5 + n], wide[:, ld - 200:ld - 72]
    _check(lowbit.lowbit_lora_accumulate(**d), *want)


def test_two_streams_with_their_own_workspaces():
    import torch

    cases = [_case(m, 1280, 3000, 32, 9, "f16", "f32", seed=m) for m in (8, 200)]
    wants = [_want(d, d["y"].cpu().double().numpy(), "f32") for d in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for d, s in zip(cases, streams):
        with torch.cuda.stream(s):
            lowbit.lowbit_lora_accumulate(**d)
    torch.cuda.synchronize()
    for d, want in zip(cases, wants):
        _check(d["y"], *want)


# rows: one launch; grouped in every work-group; sorted first
ROWS = [3, 30, 70, 200]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_small_inner_values_beside_large_ones(m, xt, yt):
    """Inner values 2^27 apart in one row, and outputs that take only the small
    ones: their products are as exact as any."""
    import torch

    g = np.random.default_rng(m)
    k, n, r = 64, 90, 40
    d = _case(m, k, n, r, 2, xt, yt, ids=np.arange(m) % 2, seed=50 + m)
    a = g.standard_normal((2, r, k))
    a[:, :24] *= 2.0 ** 13
    a[:, 24:] *= 2.0 ** -14
    b = g.standard_normal((2, n, r)) * 0.3
    b[:, ::2, :24] = 0.0
    d["a"], d["b"] = _t(a, xt), _t(b, xt)
    d["y"].zero_()
    got = lowbit.lowbit_lora_accumulate(**d)
    torch.cuda.synchronize()
    _check(got, *_want(d, np.zeros((m, n)), yt))


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_infinite_weights_follow_the_formula(m, xt, yt):
    """An infinite entry of B gives an infinity of the product's sign, whatever
    bits the inner value has; times an inner value of zero, NaN."""
    import torch

    k, n, r = 64, 70, 24
    d = _case(m, k, n, r, 2, xt, yt, ids=np.arange(m) % 2, seed=60 + m)
    d["x"][0] = 0.0
    d["x"][1] = 0.0
    d["x"][1, 5] = 1.0
    d["a"][1, 3, 5] = -2.0   # an inner value of one bit
    d["scales"][1] = 0.5
    d["x"][2] = 0.0          # a row of zeros
    d["a"][0, 20, 0] = 1.0
    d["x"][0, 0] = 1.0
    d["b"][1, 3, 3] = float("inf")
    d["b"][1, 4, 3] = -float("inf")
    d["b"][0, 64, 20] = float("inf")
    y0 = d["y"].cpu().double().numpy()
    got = lowbit.lowbit_lora_accumulate(**d).cpu().double().numpy()
    with np.errstate(invalid="ignore"):
        want, bound = _want(d, y0, yt)
    assert want[1, 3] == -np.inf and want[1, 4] == np.inf and want[0, 64] == np.inf and np.isnan(want[2, 64])
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
    assert (np.abs(got - want)[fine] <= bound[fine]).all()


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_inner_values_at_the_end_of_fp32(m, xt, yt):
    """Finite inner values that a 16-bit type rounds to infinity."""
    import torch

    d = _case(m, 8, 40, 8, 1, xt, yt, ids=np.zeros(m), seed=70 + m)
    d["x"].zero_()
    d["x"][:, 0] = 1.0
    d["a"][0, :, 0] = torch.tensor([1.0, -1.0, 0.5, 0.0, 1.0, 1.0, -0.25, 0.0])
    d["scales"][0] = 3.4e38
    d["b"] = _t(np.random.default_rng(m).uniform(1.0, 2.0, (1, 40, 8)) * 2.0 ** -14, xt)
    y0 = d["y"].cpu().double().numpy()
    _check(lowbit.lowbit_lora_accumulate(**d), *_want(d, y0, yt))


@pytest.mark.parametrize("m,k,n,r,slots", [
    (4100, 136, 300, 32, 8),      # 32 ranks to a work-group of the first product, items of 32 rows
    (4100, 136, 2049, 128, 8),    # 48 ranks; two shares of the outputs one after the other, four pieces of ranks each
    (2100, 264, 4099, 72, 5), (4100, 128, 2800, 256, 3),
    (600, 64, 5000, 72, 300),     # items of 16 rows, three shares of the outputs
    (1500, 1032, 515, 64, 20)])
@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_many_rows(m, k, n, r, slots, xt, yt):
    import torch

    say(f"lora many rows m={m} k={k} n={n} r={r} slots={slots} {xt} {yt}")
    d = _case(m, k, n, r, slots, xt, yt, ragged=True, seed=m + n)
    y0 = d["y"].clone()
    got = lowbit.lowbit_lora_accumulate(**d)
    again = lowbit.lowbit_lora_accumulate(**{**d, "y": y0.clone()})
    torch.cuda.synchronize()
    assert torch.equal(again, got)
    ids = d["ids"].cpu().numpy()
    none = torch.from_numpy((ids < 0) | (ids >= slots)).cuda()
    assert bool(none.any()) and torch.equal(got[none], y0[none])
    g = np.random.default_rng(r)
    rows = np.unique(np.concatenate([[0, m - 1], g.choice(m, 60, replace=False)]))
    part = {**d, "x": d["x"][rows], "ids": d["ids"][rows]}
    _check(got[rows], *_want(part, y0[rows].cpu().double().numpy(), yt))
    # rows in calls of few rows: the same sums in another order.  The inner values
    # are sums of some 20 in magnitudes, y's of at most 256 * 0.24 * 2 * 20 < 2500, in
    # (k / 32 + 130) + (r + 16) < 500 roundings: 0.075 for each call; another row's
    # sums would be off by more than that nearly everywhere.
    for i in range(0, m, 64 * 16):
        at = slice(i, min(i + 64, m))
        few = lowbit.lowbit_lora_accumulate(**{**d, "x": d["x"][at], "ids": d["ids"][at].contiguous(), "y": y0[at].clone()})
        off = (few.double() - got[at].double()).abs()
        step = 2.0 ** -7 if yt == "bf16" else 2.0 ** -23
        assert bool((off <= 0.15 + step * few.double().abs()).all())
