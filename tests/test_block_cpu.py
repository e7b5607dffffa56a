"""Rotary positions, the 4-bit cache, attention and sampling without a GPU:
the host-only queries, and what the C interface and the binding refuse before
any launch."""
import ctypes
import math

import numpy as np
import pytest

from bit_matmul_lowbit_amd import lowbit
from tests import plain64_block as P64

OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 6
F32, F16, BF16 = 1, 2, 3
P = ctypes.c_void_p
GOOD, OTHER, THIRD = P(0x10000), P(0x20000), P(0x30000)  # never dereferenced: every call fails validation
ODD, NULL = P(0x10001), P(0)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(lowbit.LIB_PATH):
        from bit_matmul_lowbit_amd import build

        build.build()
    return lowbit.load()


# ---------------------------------------------------------------------------
# queries

@pytest.mark.parametrize("rot,theta,scaling,factor,trained", [
    (2, 10000.0, "none", 1.0, 1), (64, 1e6, "none", 1.0, 1), (128, 10000.0, "linear", 4.0, 1), (1024, 5e5, "none", 1.0, 1),
    (128, 10000.0, "ntk", 8.0, 1), (64, 10000.0, "yarn", 16.0, 4096), (128, 1e6, "yarn", 8.0, 32768),
    (16, 10000.0, "yarn", 1.0, 8), (20, 1.5, "yarn", 3.0, 100)])
def test_turns(lib, rot, theta, scaling, factor, trained):
    turns, gain = lowbit.lowbit_rope_turns(rot, theta, scaling, factor, trained, device="cpu")
    f, want_gain = P64.frequencies(rot, theta, scaling, factor, trained)
    got = np.array([int(t) % 2 ** 64 for t in turns], dtype=object)
    want = [float(v) / (2 * math.pi) * 2.0 ** 64 for v in f]
    # a power and a few operations in FP64, and a whole number at the end
    assert all(abs(float(a) - b) <= 1 + abs(b) * 2.0 ** -45 for a, b in zip(got, want))
    assert abs(gain - want_gain) < 1e-12 and len(turns) == rot // 2


@pytest.mark.parametrize("over,status", [
    (dict(turns=None), ARG), (dict(theta=1.0), ARG), (dict(theta=float("nan")), ARG), (dict(theta=float("inf")), ARG),
    (dict(scaling=4), ARG), (dict(scaling=-1), ARG), (dict(scaling=1, factor=0.5), ARG),
    (dict(scaling=3, factor=float("inf")), ARG), (dict(scaling=3, trained=0), ARG), (dict(scaling=3, slow=0.0), ARG),
    (dict(scaling=3, fast=0.5), ARG), (dict(rot=0), SHAPE), (dict(rot=7), SHAPE), (dict(rot=1026), SHAPE),
    (dict(scaling=2, rot=2), SHAPE), (dict(), OK)])
def test_turns_refusals(lib, over, status):
    out = (ctypes.c_uint64 * 512)()
    a = dict(rot=64, theta=10000.0, scaling=0, factor=2.0, trained=4096, fast=32.0, slow=1.0, turns=out, gain=None)
    a.update(over)
    assert lib.lowbit_rope_turns(*a.values()) == status


def test_sizes(lib):
    assert lowbit.lowbit_kv_page_bytes(8, 128, 16) == 8 * 16 * 160
    assert lowbit.lowbit_kv_page_bytes(4, 256, 64) == 4 * 64 * 320
    # 64 KiB a token in FP16 over 16 layers of 4 heads of 256: 20 KiB here
    assert 16 * lowbit.lowbit_kv_page_bytes(4, 256, 16) // 16 == 64 * 1024 * 5 // 16
    for bad in ((0, 128, 16), (1025, 128, 16), (8, 96, 16), (8, 128, 8), (8, 128, 24), (8, 128, 512), (-1, 128, 16)):
        assert lowbit.lowbit_kv_page_bytes(*bad) == 0
    for good in ((1, 1, 16, 8, 128, 1), (6144, 3, 32, 8, 128, 2048), (61, 61, 24, 4, 256, 1), (5, 2, 7, 1, 64, 4)):
        assert lowbit.lowbit_attention_workspace_bytes(*good) > 0
    for bad in ((0, 1, 16, 8, 128, 1), (1, 0, 16, 8, 128, 1), (1, 1, 15, 8, 128, 1), (1, 1, 16, 8, 96, 1),
                (1, 1, 16, 8, 128, 0), (1, 1, 0, 0, 128, 1), (1, 1, 2048, 8, 128, 1), (1, 65536, 16, 8, 128, 1)):
        assert lowbit.lowbit_attention_workspace_bytes(*bad) == 0
    assert lowbit.lowbit_sample_workspace_bytes(151936, 64) > 0 == lowbit.lowbit_sample_workspace_bytes(0, 1)
    assert lowbit.lowbit_sample_workspace_bytes((1 << 20) + 1, 1) == 0 == lowbit.lowbit_sample_workspace_bytes(5, 65536)


# ---------------------------------------------------------------------------
# refusals of the C interface

ROPE = dict(x=GOOD, xt=F16, ldx=512, ldxh=128, pos=GOOD, turns=GOOD, m=2, heads=4, d=128, rot=64, inter=0, gain=1.0,
            out=OTHER, ot=F16, ldo=512, ldoh=128, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(x=NULL), ARG), (dict(pos=NULL), ARG), (dict(turns=NULL), ARG), (dict(out=NULL), ARG), (dict(xt=0), ARG),
    (dict(ot=5), ARG), (dict(gain=float("nan")), ARG), (dict(gain=float("inf")), ARG), (dict(out=GOOD, ot=F32), ARG),
    (dict(out=GOOD, ldo=600), ARG), (dict(out=GOOD, ldoh=130, ldo=600, ldx=600), ARG),
    (dict(m=0), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE),
    (dict(d=1026, rot=64), SHAPE), (dict(d=1), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE),
    (dict(rot=130), SHAPE), (dict(ldx=511), SHAPE), (dict(ldxh=127), SHAPE), (dict(ldo=511), SHAPE), (dict(ldoh=-128), SHAPE),
    (dict(ldx=128, ldxh=200), SHAPE), (dict(ldx=1 << 62), SHAPE), (dict(ldxh=1 << 62), SHAPE),
    (dict(x=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(xt=F32, x=P(0x10002)), ALIGN), (dict(pos=P(0x10002)), ALIGN),
    (dict(turns=P(0x10004)), ALIGN)])
def test_rope_refusals(lib, over, status):
    assert lib.lowbit_rope(*{**ROPE, **over}.values()) == status


STORE = dict(k=GOOD, ldk=512, ldkh=128, v=GOOD, ldv=512, ldvh=128, type=F16, slots=GOOD, m=2, heads=4, d=128, pages=OTHER,
             n=10, page=16, pos=GOOD, turns=GOOD, rot=64, inter=0, gain=1.0, q=GOOD, ldq=1024, ldqh=128, hq=8, qo=THIRD,
             qt=F16, ldqo=1024, ldqoh=128, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(slots=NULL), ARG), (dict(pages=NULL), ARG), (dict(type=0), ARG),
    (dict(pos=NULL), ARG), (dict(turns=NULL), ARG), (dict(pos=NULL, turns=NULL), ARG), (dict(qo=NULL), ARG),
    (dict(q=NULL), ARG), (dict(qt=0), ARG), (dict(gain=float("nan")), ARG), (dict(qo=GOOD, qt=BF16), ARG),
    (dict(qo=GOOD, ldqo=1025), ARG),
    (dict(m=0), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(d=96), SHAPE),
    (dict(d=512), SHAPE), (dict(n=0), SHAPE), (dict(n=1 << 27), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE),
    (dict(page=512), SHAPE), (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(ldk=500), SHAPE),
    (dict(ldvh=100), SHAPE), (dict(hq=0), SHAPE), (dict(hq=1025), SHAPE), (dict(ldq=1023), SHAPE), (dict(ldqo=1), SHAPE),
    (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(slots=P(0x10002)), ALIGN), (dict(pages=P(0x20008)), ALIGN),
    (dict(pos=P(0x10002)), ALIGN), (dict(turns=P(0x10004)), ALIGN), (dict(q=ODD), ALIGN), (dict(qo=P(0x30001)), ALIGN),
    (dict(qt=F32, qo=P(0x30002)), ALIGN)])
def test_store_refusals(lib, over, status):
    assert lib.lowbit_kv_store(*{**STORE, **over}.values()) == status


LOAD = dict(pages=GOOD, n=10, heads=4, d=128, page=16, slots=GOOD, m=2, k=OTHER, ldk=512, ldkh=128, v=THIRD, ldv=512,
            ldvh=128, type=F16, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(pages=NULL), ARG), (dict(slots=NULL), ARG), (dict(k=NULL, v=NULL), ARG), (dict(type=4), ARG), (dict(v=OTHER), ARG),
    (dict(m=0), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(heads=0), SHAPE), (dict(d=32), SHAPE), (dict(page=17), SHAPE),
    (dict(n=0), SHAPE), (dict(ldk=511), SHAPE), (dict(ldvh=1), SHAPE),
    (dict(pages=P(0x10004)), ALIGN), (dict(slots=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(type=F32, v=P(0x30002)), ALIGN)])
def test_load_refusals(lib, over, status):
    assert lib.lowbit_kv_load(*{**LOAD, **over}.values()) == status


ATTN = dict(q=GOOD, qt=F16, ldq=1024, ldqh=128, m=2, hq=8, pages=GOOD, n=10, heads=4, d=128, page=16, table=GOOD, tcap=5,
            ldt=5, lengths=GOOD, qs=NULL, b=2, max_q=1, scale=0.1, out=OTHER, ot=F16, ldo=1024, ldoh=128, lse=NULL,
            ws=THIRD, wsb=1 << 30, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(q=NULL), ARG), (dict(pages=NULL), ARG), (dict(table=NULL), ARG), (dict(lengths=NULL), ARG), (dict(out=NULL), ARG),
    (dict(qt=F32), ARG), (dict(ot=0), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
    (dict(out=GOOD), ARG), (dict(m=3), ARG), (dict(max_q=2), ARG),
    (dict(m=0, b=0), SHAPE), (dict(qs=GOOD, m=(1 << 22) + 1), SHAPE), (dict(m=65536, b=65536), SHAPE),
    (dict(qs=GOOD, max_q=0), SHAPE), (dict(hq=9), SHAPE), (dict(hq=2), SHAPE), (dict(hq=1028), SHAPE), (dict(d=80), SHAPE),
    (dict(page=20), SHAPE), (dict(n=0), SHAPE), (dict(tcap=0), SHAPE), (dict(ldt=4), SHAPE),
    (dict(tcap=(1 << 26) + 1, ldt=1 << 27), SHAPE), (dict(ldq=1000), SHAPE), (dict(ldoh=64), SHAPE),
    (dict(q=ODD), ALIGN), (dict(pages=P(0x10008)), ALIGN), (dict(table=P(0x10002)), ALIGN), (dict(lengths=ODD), ALIGN),
    (dict(qs=ODD), ALIGN), (dict(out=P(0x20001)), ALIGN), (dict(lse=P(0x20002)), ALIGN), (dict(ws=P(0x30008)), ALIGN),
    (dict(ws=NULL), WS), (dict(wsb=64), WS)])
def test_attention_refusals(lib, over, status):
    assert lib.lowbit_attention(*{**ATTN, **over}.values()) == status


SAMPLE = dict(y=GOOD, yt=F32, ldy=100, n=100, b=2, t=GOOD, k=GOOD, p=GOOD, mp=GOOD, u=GOOD, idx=OTHER, prob=OTHER, ws=THIRD,
              wsb=1 << 20, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(y=NULL), ARG), (dict(u=NULL), ARG), (dict(idx=NULL), ARG), (dict(yt=7), ARG),
    (dict(n=0), SHAPE), (dict(n=(1 << 20) + 1, ldy=1 << 21), SHAPE), (dict(b=0), SHAPE), (dict(b=65536), SHAPE),
    (dict(ldy=99), SHAPE), (dict(ldy=1 << 62), SHAPE),
    (dict(y=P(0x10002)), ALIGN), (dict(t=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(p=ODD), ALIGN), (dict(mp=ODD), ALIGN),
    (dict(u=ODD), ALIGN), (dict(idx=P(0x20002)), ALIGN), (dict(prob=P(0x20002)), ALIGN), (dict(ws=P(0x30004)), ALIGN),
    (dict(ws=NULL), WS), (dict(wsb=100), WS)])
def test_sample_refusals(lib, over, status):
    assert lib.lowbit_sample(*{**SAMPLE, **over}.values()) == status


# ---------------------------------------------------------------------------
# the binding

def test_the_compiled_functions_count_their_arguments():
    from bit_matmul_lowbit_amd import _marshal

    for f in (_marshal.rope, _marshal.kv_store, _marshal.kv_load, _marshal.attention, _marshal.sample):
        with pytest.raises(TypeError, match="expected"):
            f("name")


@pytest.mark.parametrize("call", [
    lambda t: lowbit.lowbit_rope(t(1, 2, 64), t(1), t(32)),
    lambda t: lowbit.lowbit_rope([1.0], t(1), t(32)),
    lambda t: lowbit.lowbit_rope(t(1, 2, 64), t(1), t(32), out_dtype="float16"),
    lambda t: lowbit.lowbit_kv_store(t(1, 2, 64), t(1, 2, 64), t(1), t(1, 2560), 16),
    lambda t: lowbit.lowbit_kv_store(t(1, 2, 64), t(1, 2, 64), t(1), None, 16),
    lambda t: lowbit.lowbit_kv_load(t(1, 2560), 16, t(1), 2, 64),
    lambda t: lowbit.lowbit_kv_load(None, 16, t(1), 2, 64),
    lambda t: lowbit.lowbit_attention(t(1, 2, 64), t(1, 2560), 16, t(1, 1), t(1)),
    lambda t: lowbit.lowbit_attention(3, t(1, 2560), 16, t(1, 1), t(1)),
    lambda t: lowbit.lowbit_sample(t(1, 100), t(1)),
    lambda t: lowbit.lowbit_sample([1.0], t(1)),
])
def test_host_tensors_and_other_objects_are_refused(call):
    import torch

    with pytest.raises(TypeError):
        call(torch.zeros)


def test_unknown_scaling_is_refused():
    with pytest.raises(KeyError):
        lowbit.lowbit_rope_turns(64, scaling="cubic", device="cpu")
    with pytest.raises(lowbit.LowbitError):
        lowbit.lowbit_rope_turns(63, device="cpu")
    with pytest.raises(lowbit.LowbitError):
        lowbit.lowbit_rope_turns(-4, device="cpu")
