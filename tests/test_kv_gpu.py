"""Rotary positions and the 4-bit cache on the GPU against tests/plain64_block.py:
angles, layouts, strides, types, slots; bytes of the cache bit for bit."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P
from tests.helpers import say

pytestmark = pytest.mark.gpu

NAMES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def dt(name):
    import torch

    return getattr(torch, NAMES[name])


def dev(a, name="f32"):
    """numpy -> GPU tensor of that type, and the values it then has"""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dt(name)).cuda()
    return t, t.float().cpu().numpy()


def i32(a):
    import torch

    return torch.tensor(np.asarray(a).tolist(), dtype=torch.int32, device="cuda")


def host(t):
    return t.double().cpu().numpy()


def turns_of(rot, **kw):
    t, gain = lowbit.lowbit_rope_turns(rot, **kw)
    return t, [int(v) % 2 ** 64 for v in t], gain


POSITIONS = [0, 1, 262143, 2 ** 31 - 1, -1, -2 ** 31, 4097, 31]


@pytest.mark.parametrize("x,out", [("f32", "f16"), ("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("m,heads,d,rot", [(1, 1, 2, 2), (1, 16, 128, 128), (8, 24, 256, 64), (8, 3, 80, 36), (5, 7, 106, 4),
                                           (8, 1, 1024, 1024), (3, 2, 30, 30), (6, 40, 64, 16)])
def test_rope(x, out, inter, m, heads, d, rot):
    say("rope", x, out, inter, m, heads, d, rot)
    g = np.random.default_rng(m * 1000 + d)
    t, turns, gain = turns_of(rot, theta=1e6, scaling="yarn", factor=8.0, trained=32768)
    xt, xv = dev(g.standard_normal((m, heads, d)) * 3, x)
    pos = POSITIONS[:m]
    got = lowbit.lowbit_rope(xt, i32(pos), t, interleaved=inter, gain=gain, out_dtype=dt(out))
    assert got.dtype == dt(out)
    want = P.rope(xv, pos, turns, inter, gain)
    assert (np.abs(host(got) - want) <= P.rope_bound(xv, pos, turns, inter, gain, NAMES[out])).all()
    if out == "f32":  # what does not turn is copied
        assert np.array_equal(got[..., rot:].cpu().numpy(), xv[..., rot:])


@pytest.mark.parametrize("m,heads,d,rot", [(1000, 8, 128, 128), (4099, 3, 96, 32), (257, 40, 64, 62), (20000, 1, 64, 64)])
def test_rope_many_rows_in_place_and_strided(m, heads, d, rot):
    import torch

    say("rope rows", m, heads, d, rot)
    g = np.random.default_rng(m)
    t, turns, _ = turns_of(rot)
    wide, values = dev(g.standard_normal((m, heads + 2, d + 3)), "bf16")
    pos = g.integers(0, 262144, m)
    for inter in (False, True):
        before = wide.clone()
        x = wide[:, 1:1 + heads, 3:]  # odd offsets and strides
        want = P.rope(values[:, 1:1 + heads, 3:], pos, turns, inter)
        bound = P.rope_bound(values[:, 1:1 + heads, 3:], pos, turns, inter, 1.0, "bfloat16")
        apart = lowbit.lowbit_rope(x, i32(pos), t, interleaved=inter)
        assert (np.abs(host(apart) - want) <= bound).all()
        # heads before tokens
        by_head = torch.empty(heads, m, d, dtype=torch.bfloat16, device="cuda")
        lowbit.lowbit_rope(x, i32(pos), t, interleaved=inter, out=by_head.transpose(0, 1))
        assert torch.equal(by_head.transpose(0, 1), apart)
        assert lowbit.lowbit_rope(x, i32(pos), t, interleaved=inter, out=x) is x
        assert torch.equal(x, apart)
        x.copy_(before[:, 1:1 + heads, 3:])
        assert torch.equal(wide, before)  # nothing beside it was written


def test_rope_what_is_not_finite_stays_in_its_pair():
    import torch

    t, turns, _ = turns_of(64)
    x = torch.ones(2, 1, 64, device="cuda")
    x[0, 0, 3], x[1, 0, 40] = float("inf"), float("nan")
    y = lowbit.lowbit_rope(x, i32([5, 6]), t)
    bad = ~torch.isfinite(y)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 35] and bad[1, 0].nonzero().flatten().tolist() == [8, 40]


# ---------------------------------------------------------------------------
# the cache

def kv(g, m, heads, d, kind):
    k, v = g.standard_normal((2, m, heads, d))
    if kind == "wide":  # channels that stand out, offsets, all scales
        k = k * 10.0 ** g.uniform(-6, 4, (m, heads, 1)) + 5 * g.standard_normal((1, heads, d))
        v = v * 10.0 ** g.uniform(-9, 3, (m, heads, 1))
    elif kind == "grid":  # ties everywhere
        k, v = np.rint(k * 4), np.rint(v * 2) / 2
    elif kind == "flat":
        k, v = np.broadcast_to(k[..., :1], k.shape), np.zeros_like(v)
    return k.astype(np.float32), v.astype(np.float32)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "wide", "grid", "flat"])
@pytest.mark.parametrize("m,heads,d,page", [(1, 8, 128, 16), (3, 1, 64, 16), (61, 4, 256, 64), (130, 3, 64, 32),
                                            (515, 2, 128, 256)])
def test_store_writes_the_bytes_of_the_definition(x, kind, m, heads, d, page):
    import torch

    say("store", x, kind, m, heads, d, page)
    g = np.random.default_rng(m + d)
    k, v = kv(g, m, heads, d, kind)
    (kt, kv_), (vt, vv) = dev(k, x), dev(v, x)
    n = m // page + 3
    fill = g.integers(0, 256, (n, P.page_bytes(heads, d, page))).astype(np.uint8)
    # in order from a multiple of four, in order from another place, anywhere, some outside
    for order in ("aligned", "shifted", "mixed"):
        slots = {"aligned": page + np.arange(m), "shifted": 3 + np.arange(m),
                 "mixed": g.permutation(n * page)[:m]}[order].astype(np.int64)
        if order == "mixed":
            slots[::7] = [-1, n * page, 2 ** 31 - 1, -2 ** 31][m % 4]
        pages = torch.from_numpy(fill.copy()).cuda()
        assert lowbit.lowbit_kv_store(kt, vt, i32(slots), pages, page) is None
        want = fill.copy()
        P.put(want, heads, d, page, slots, kv_, vv)
        got = pages.cpu().numpy()
        assert np.array_equal(got, want), (order, np.argwhere(got != want)[:5])
        for name in ("f16", "bf16", "f32"):
            kk, vv2 = lowbit.lowbit_kv_load(pages, page, i32(slots), heads, d, dtype=dt(name))
            wk, wv = (torch.from_numpy(t).to(dt(name)) for t in P.get(want, heads, d, page, slots))
            assert torch.equal(kk.cpu(), wk) and torch.equal(vv2.cpu(), wv)


def test_the_cache_holds_nothing_that_is_not_finite():
    import torch

    m, heads, d, page = 6, 2, 128, 16
    k = torch.randn(m, heads, d, device="cuda")
    k[0, 0, 5], k[1, 1, 40], k[2, 0, 100], k[3] = float("nan"), float("inf"), -float("inf"), float("nan")
    k[4, 0], k[4, 1] = 1e38, -1e38
    k[5, 0, ::2], k[5, 0, 1::2] = 3e38, -3e38
    v = k.flip(0).contiguous()
    pages = torch.full((2, P.page_bytes(heads, d, page)), 255, dtype=torch.uint8, device="cuda")
    slots = i32([0, 1, 2, 3, 17, 30])
    lowbit.lowbit_kv_store(k, v, slots, pages, page)
    want = torch.full(pages.shape, 255, dtype=torch.uint8).numpy()
    P.put(want, heads, d, page, slots.tolist(), k.cpu().numpy(), v.cpu().numpy())
    assert np.array_equal(pages.cpu().numpy(), want)
    for t in lowbit.lowbit_kv_load(pages, page, slots, heads, d):
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("x,qo", [("f32", "f16"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("m,hq,heads,d,page,rot", [(1, 16, 8, 128, 16, 128), (61, 24, 4, 256, 64, 64), (5, 1, 1, 64, 16, 16),
                                                   (1030, 5, 5, 128, 32, 96)])
def test_store_turns_keys_and_queries(inter, x, qo, m, hq, heads, d, page, rot):
    import torch

    say("store turned", inter, x, qo, m, hq, heads, d, page, rot)
    g = np.random.default_rng(m + d)
    t, turns, gain = turns_of(rot, theta=1e6, scaling="yarn", factor=4.0, trained=8192)
    # one fused product's rows, q first
    fused, values = dev(g.standard_normal((m, hq + 2 * heads, d)), x)
    q, k, v = fused[:, :hq], fused[:, hq:hq + heads], fused[:, hq + heads:]
    pos = g.integers(0, 262144, m)
    n = m // page + 2
    slots = np.arange(m) + 4
    pages = torch.zeros(n, P.page_bytes(heads, d, page), dtype=torch.uint8, device="cuda")
    got_q = lowbit.lowbit_kv_store(k, v, i32(slots), pages, page, positions=i32(pos), turns=t, interleaved=inter,
                                   gain=gain, q=q, q_dtype=dt(qo))
    qv, kv_, vv = values[:, :hq], values[:, hq:hq + heads], values[:, hq + heads:]
    assert (np.abs(host(got_q) - P.rope(qv, pos, turns, inter, gain)) <=
            P.rope_bound(qv, pos, turns, inter, gain, NAMES[qo])).all()
    # alone it is the same
    assert torch.equal(got_q, lowbit.lowbit_rope(q, i32(pos), t, interleaved=inter, gain=gain, out_dtype=dt(qo)))
    kk, vv2 = lowbit.lowbit_kv_load(pages, page, i32(slots), heads, d)
    assert np.array_equal(vv2.cpu().numpy(), P.held(vv))
    # FP32 turned keys, held in 4 bits: within what 4 bits take, and what FP32 takes from the keys
    turned = P.rope(kv_, pos, turns, inter, gain)
    bound = P.held_bound(turned) * (1 + 1e-5) + P.rope_bound(kv_, pos, turns, inter, gain, "float32") * 2
    assert (np.abs(host(kk) - turned) <= bound).all()
    # and what the turned keys of their own, stored as they come, give
    other = torch.zeros_like(pages)
    exact = lowbit.lowbit_rope(k, i32(pos), t, interleaved=inter, gain=gain, out_dtype=torch.float32)
    lowbit.lowbit_kv_store(exact, v.float(), i32(slots), other, page)
    assert torch.equal(pages, other)
    # in place
    fresh = fused.clone()
    if x == qo:
        qq = fresh[:, :hq]
        assert lowbit.lowbit_kv_store(fresh[:, hq:hq + heads], fresh[:, hq + heads:], i32(slots), other, page,
                                      positions=i32(pos), turns=t, interleaved=inter, gain=gain, q=qq, q_out=qq) is qq
        assert torch.equal(qq, got_q) and torch.equal(fresh[:, hq:], fused[:, hq:]) and torch.equal(pages, other)


def test_load_one_of_the_two_strided_and_repeated():
    import torch

    g = np.random.default_rng(8)
    heads, d, page, m = 3, 64, 16, 40
    k, v = kv(g, m, heads, d, "plain")
    pages = torch.zeros(4, P.page_bytes(heads, d, page), dtype=torch.uint8, device="cuda")
    lowbit.lowbit_kv_store(dev(k)[0], dev(v)[0], i32(np.arange(m)), pages, page)
    slots = [7, 7, 7, 7, 0, 63, 64, -5, 12, 13, 14, 15, 16, 17]
    wk, wv = P.get(pages.cpu().numpy(), heads, d, page, slots)
    wide = torch.full((heads, len(slots), d + 8), 9.0, dtype=torch.float16, device="cuda")
    out = wide[:, :, 1:1 + d].transpose(0, 1)
    got = lowbit.lowbit_kv_load(pages, page, i32(slots), heads, d, v_out=out)
    assert got[0] is None and np.array_equal(out.cpu().numpy(), wv)
    assert (wide[:, :, 0] == 9).all() and (wide[:, :, 1 + d:] == 9).all()
    got = lowbit.lowbit_kv_load(pages, page, i32(slots), heads, d, k_out=out)
    assert got[1] is None and np.array_equal(out.cpu().numpy(), wk)


def test_a_cache_past_32_bits_of_bytes():
    """5.4 GB of pages: the last page is as good as the first."""
    import torch

    heads, d, page = 4, 256, 64
    one = P.page_bytes(heads, d, page)
    n = 5_400_000_000 // one
    g = np.random.default_rng(9)
    k, v = kv(g, 6, heads, d, "plain")
    pages = torch.empty(n, one, dtype=torch.uint8, device="cuda")
    pages[-2:] = 0
    slots = (n - 2) * page + np.array([0, 1, 2, 3, 70, 127])
    lowbit.lowbit_kv_store(dev(k)[0], dev(v)[0], i32(slots), pages, page)
    kk, vv = lowbit.lowbit_kv_load(pages, page, i32(slots), heads, d)
    assert np.array_equal(kk.cpu().numpy(), P.held(k)) and np.array_equal(vv.cpu().numpy(), P.held(v))
    want = np.zeros((2, one), np.uint8)
    P.put(want, heads, d, page, slots - (n - 2) * page, k, v)
    assert np.array_equal(pages[-2:].cpu().numpy(), want)
