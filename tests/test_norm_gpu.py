"""lowbit_norm_residual against its plain form in 64 bits: both norms and none
on either side of the residual, gates, every type, widths from one element to
past what a work-group keeps in registers, strided and unaligned rows."""
import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64
from tests.helpers import GUARD_BYTE, guarded, guards_intact, say

pytestmark = pytest.mark.gpu

NAMES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def _make(g, shape, name, sigma=1.0, mean=0.0):
    """(device tensor of the type, its values in 64 bits)"""
    import torch

    t = torch.from_numpy(g.standard_normal(shape) * sigma + mean).to(getattr(torch, NAMES[name])).cuda()
    return t, t.cpu().double().numpy()


def _vec(g, k, sigma, mean):
    import torch

    t = torch.from_numpy((g.standard_normal(k) * sigma + mean).astype(np.float32)).cuda()
    return t, t.cpu().double().numpy()


def _case(m, k, yt, rt, xt, post, pre, gate, seed, mean=0.0, eps=1e-6, weights=True):
    g = np.random.default_rng(seed)
    d = dict(m=m, k=k, yt=yt, rt=rt, xt=xt, post=post, pre=pre, eps=eps, scale=0.375)
    d["y"] = _make(g, (m, k), yt, 2.0, mean)
    d["r"] = _make(g, (m, k), rt, 3.0, mean)
    none = (None, None)
    for side, kind in (("post", post), ("pre", pre)):
        d[side + "_w"] = _vec(g, k, 0.2, 1.0) if kind != "none" and weights else none
        d[side + "_b"] = _vec(g, k, 0.2, 0.0) if kind == "layer" and weights else none
    d["gate"] = {"none": lambda: none, "channel": lambda: _make(g, (k,), "f32", 0.3, 0.7),
                 "row": lambda: _make(g, (m, k), "f32", 0.3, 0.7),
                 "row_bf16": lambda: _make(g, (m, k), "bf16", 0.3, 0.7)}[gate]()
    return d


def _call(d, **over):
    import torch

    args = dict(post=d["post"], post_w=d["post_w"][0], post_b=d["post_b"][0], gate=d["gate"][0],
                scale=d["scale"], pre=d["pre"], pre_w=d["pre_w"][0], pre_b=d["pre_b"][0], eps=d["eps"],
                x_dtype=getattr(torch, NAMES[d["xt"]]))
    args.update(over)
    return lowbit.lowbit_norm_residual(over.pop("y", d["y"][0]), args.pop("r", d["r"][0]),
                                       **{k: v for k, v in args.items() if k != "y"})


def _want(d):
    a = (d["y"][1], d["r"][1], d["post"], d["post_w"][1], d["post_b"][1], d["gate"][1], d["scale"], d["pre"],
         d["pre_w"][1], d["pre_b"][1], d["eps"])
    return plain64.norm_residual(*a), plain64.norm_residual_bound(*a, NAMES[d["rt"]], NAMES[d["xt"]])


def _check(d, r_out, x_out):
    (rr, x), (er, ex) = _want(d)
    for got, want, err, what in ((r_out, rr, er, "r"), (x_out, x, ex, "x")):
        got = got.cpu().double().numpy()
        off = np.abs(got - want) - err
        assert np.isfinite(got).all() and off.max() <= 0, \
            f"{what}: off by {np.abs(got - want).max():.3g}, over its bound by {off.max():.3g}"


SHAPES = [(1, 1), (1, 2048), (3, 127), (5, 128), (7, 1283), (4, 5120), (2, 8193), (3, 8200), (1, 17408),
          (2, 40000), (300, 640), (70, 5120)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("post,pre,gate", [("none", "rms", "none"), ("rms", "rms", "row"),
                                           ("layer", "layer", "channel")])
def test_matches_plain_form(m, k, post, pre, gate):
    import torch

    say(f"norm m={m} k={k} {post} {pre} {gate}")
    d = _case(m, k, "f32", "f32", "f16", post, pre, gate, 100 + m + k)
    r_out = torch.empty_like(d["r"][0])
    before = d["r"][0].clone()
    got = _call(d, r_out=r_out)
    torch.cuda.synchronize()
    assert got[0] is r_out and torch.equal(d["r"][0], before)
    _check(d, *got)


@pytest.mark.parametrize("m,k", [(1024, 7), (1500, 8), (1031, 9), (9000, 128), (5003, 511), (4100, 514), (5000, 1001),
                                 (4300, 1025), (1100, 4095), (700, 4096), (1100, 5119), (1030, 8200),
                                 (1100, 640), (1030, 1024), (1500, 1032), (1100, 4096), (1024, 12296)])
@pytest.mark.parametrize("yt,rt,xt", [("f32", "f32", "f16"), ("bf16", "bf16", "bf16"), ("f16", "f32", "bf16")])
@pytest.mark.parametrize("post,pre,gate,pad", [("none", "none", "none", 0), ("rms", "rms", "none", 3),
                                               ("layer", "layer", "channel", 0), ("rms", "layer", "row", 8)])
def test_many_rows(m, k, yt, rt, xt, post, pre, gate, pad):
    """Work-groups and waves that take several rows and keep the weights, in
    place and not, at row strides of their own."""
    import torch

    say(f"norm m={m} k={k} y={yt} r={rt} x={xt} {post} {pre} {gate} pad={pad}")
    d = _case(m, k, yt, rt, xt, post, pre, gate, m + k + pad)
    wide = torch.full((m + 1, k + pad), 77.0, dtype=d["r"][0].dtype, device="cuda")
    r = wide[:m, :k]
    r.copy_(d["r"][0])
    r_out, x_out = _call(d, r=r)
    torch.cuda.synchronize()
    assert r_out is r
    _check(d, r_out, x_out)
    assert bool((wide[:m, k:] == 77.0).all()) and bool((wide[m] == 77.0).all())
    r2 = torch.empty_like(d["r"][0])
    _, x2 = _call(d, r_out=r2)
    assert torch.equal(r2, r_out) and torch.equal(x2, x_out)


@pytest.mark.parametrize("yt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(3, 1280), (33, 331)])
def test_types_in_place(yt, rt, xt, m, k):
    import torch

    say(f"norm types y={yt} r={rt} x={xt} m={m} k={k}")
    d = _case(m, k, yt, rt, xt, "rms", "layer", "row_bf16" if xt == "bf16" else "channel", 7 * m)
    r0 = d["r"][0].clone()
    r_out, x_out = _call(d)
    torch.cuda.synchronize()
    assert r_out is d["r"][0]
    _check(d, r_out, x_out)
    # the same inputs give the same bits, in place or not
    r2 = torch.empty_like(r0)
    _, x2 = _call(d, r=r0, r_out=r2)
    assert torch.equal(r2, r_out) and torch.equal(x2, x_out)


@pytest.mark.parametrize("k", [5120, 1001])
def test_large_mean_and_no_weights(k):
    d = _case(4, k, "f32", "f32", "f32", "layer", "layer", "none", 5, mean=1000.0, weights=False)
    _check(d, *_call(d))
    d = _case(4, k, "bf16", "bf16", "bf16", "rms", "rms", "none", 6, mean=50.0, weights=False)
    _check(d, *_call(d))


def test_parts_alone():
    import torch

    d = _case(5, 1280, "bf16", "f32", "f16", "rms", "rms", "none", 8)
    # only the norm of r
    r0 = d["r"][0].clone()
    got, x = lowbit.lowbit_norm_residual(None, d["r"][0], pre="rms", pre_w=d["pre_w"][0])
    want = plain64.norm(d["r"][1], "rms", d["pre_w"][1])
    assert got is d["r"][0] and torch.equal(got, r0) and x.dtype == torch.float16
    err = np.abs(x.cpu().double().numpy() - want)
    assert (err <= plain64.rounding(want, "float16") + 1e-5).all()
    # only the residual
    got, x = lowbit.lowbit_norm_residual(d["y"][0], d["r"][0], post="rms", post_w=d["post_w"][0], scale=0.5)
    assert x is None
    want, _ = plain64.norm_residual(d["y"][1], d["r"][1], "rms", d["post_w"][1], scale=0.5)
    assert (np.abs(got.cpu().double().numpy() - want) <= 1e-5 * (1 + np.abs(want))).all()
    # neither norm: the sum, cast
    got, x = lowbit.lowbit_norm_residual(d["y"][0], d["r"][0].copy_(r0), pre="none", x_dtype=torch.bfloat16)
    assert torch.equal(got, r0 + d["y"][0].float()) and torch.equal(x, got.to(torch.bfloat16))


def test_zero_and_bad_rows():
    import torch

    d = _case(4, 384, "f32", "f32", "f16", "rms", "rms", "none", 9)
    y, r = d["y"][0], d["r"][0]
    y[0] = 0.0
    r[0] = 0.0
    y[1, 5] = float("inf")
    r[2, 7] = float("nan")
    r_out, x = _call(d)
    assert not r_out[0].any() and not x[0].any()
    assert not torch.isfinite(x[1]).all() and torch.isnan(x[2]).all()
    d["y"], d["r"] = (y, y.cpu().double().numpy()), d["r"]
    (rr, xx), (er, ex) = _want(d)
    assert (np.abs(r_out[3].cpu().double().numpy() - rr[3]) <= er[3]).all()
    assert (np.abs(x[3].cpu().double().numpy() - xx[3]) <= ex[3]).all()


@pytest.mark.parametrize("off,pad", [(0, 64), (8, 24), (1, 7), (3, 0)])
def test_strided_and_unaligned_rows(off, pad):
    import torch

    say(f"norm strided off={off} pad={pad}")
    m, k = 6, 1280
    d = _case(m, k, "bf16", "f16", "f16", "layer", "rms", "row", 11)

    def wide(t):
        buf = torch.full((m, off + k + pad), 77.0, dtype=t.dtype, device="cuda")
        buf[:, off:off + k] = t
        return buf, buf[:, off:off + k]

    yb, y = wide(d["y"][0])
    rb, r = wide(d["r"][0])
    gb, gate = wide(d["gate"][0])
    xb, x = wide(torch.zeros(m, k, dtype=torch.float16, device="cuda"))
    got = _call(d, y=y, r=r, gate=gate, x_out=x)
    torch.cuda.synchronize()
    _check(d, *got)
    for buf in (rb, xb):  # nothing beside the rows was written
        side = torch.cat([buf[:, :off], buf[:, off + k:]], 1)
        assert bool((side == 77.0).all())


@pytest.mark.parametrize("m,k", [(3, 1280), (2, 1003), (5, 40000)])
def test_guards_around_outputs(m, k):
    import torch

    d = _case(m, k, "f32", "f32", "f16", "rms", "rms", "none", 12)
    rraw, r_out = guarded((m + 2, k), torch.float32)
    xraw, x_out = guarded((m + 2, k), torch.float16)
    _call(d, r_out=r_out[:m], x_out=x_out[:m])
    torch.cuda.synchronize()
    _check(d, r_out[:m], x_out[:m])
    assert guards_intact(rraw) and guards_intact(xraw)
    for t in (r_out, x_out):  # rows behind the last
        assert bool((t[m:].view(torch.uint8) == GUARD_BYTE).all())


def test_graph_and_stream():
    import torch

    d = _case(8, 5120, "f32", "f32", "f16", "rms", "rms", "row", 13)
    r_out, x_out = torch.empty_like(d["r"][0]), torch.empty(8, 5120, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _call(d, r_out=r_out, x_out=x_out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(d, r_out, x_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(d, r_out=r_out, x_out=x_out)
    for _ in range(3):
        r_out.fill_(7.0)
        x_out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        _check(d, r_out, x_out)


def test_offsets_past_32_bits():
    import torch

    m, k, ld = 40, 1280, (1 << 27) + 8  # 40 rows: 5.4e9 elements, 10.7 GB
    d = _case(m, k, "f16", "f16", "f16", "rms", "layer", "channel", 15)
    wide = torch.empty(m, ld, dtype=torch.float16, device="cuda")
    places = {"y": 8, "r": 1 << 20, "x": ld - k - 1}
    y, r, x = (wide[:, o:o + k] for o in places.values())
    y.copy_(d["y"][0])
    r.copy_(d["r"][0])
    got = _call(d, y=y, r=r, x_out=x)
    _check(d, *got)


@pytest.mark.parametrize("k", [640, 40000])
def test_c_interface_copies_the_residual_without_y(k):
    """y NULL: r' is r, and goes to r_out where that is given."""
    import torch

    r = torch.randn(3, k, device="cuda")
    r_out = torch.full_like(r, 7.0)
    x = torch.empty(3, k, dtype=torch.float16, device="cuda")
    args = (None, 0, 0, r.data_ptr(), 1, k, r_out.data_ptr(), k, x.data_ptr(), 2, k, 3, k, 0, None, None, None, 0, 0, 1.0,
            1, None, None, 1e-6, torch.cuda.current_stream().cuda_stream)
    assert lowbit.load().lowbit_norm_residual(*args) == 0
    torch.cuda.synchronize()
    assert torch.equal(r_out, r)
    want = plain64.norm(r.cpu().double().numpy(), "rms")
    assert (np.abs(x.cpu().double().numpy() - want) <= plain64.rounding(want, "float16") + 1e-5).all()
