"""Refusals of the operators beside the products, on the host before any
launch (no GPU): the C interface's statuses and the binding's errors."""
import ctypes

import pytest

from bit_matmul_lowbit_amd import lowbit

OK, ARG, SHAPE, ALIGN, WS = 0, 1, 2, 3, 6
F32, F16, BF16 = 1, 2, 3
P = ctypes.c_void_p
GOOD, OTHER, THIRD = P(0x10000), P(0x20000), P(0x30000)  # never dereferenced: every call fails validation
NULL = P(0)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(lowbit.LIB_PATH):
        from bit_matmul_lowbit_amd import build

        build.build()
    return lowbit.load()


NORM = dict(y=GOOD, yt=F32, ldy=128, r=OTHER, rt=F32, ldr=128, ro=OTHER, ldro=128, x=THIRD, xt=F16, ldx=128, m=2,
            k=128, post=1, pw=NULL, pb=NULL, gate=NULL, gt=0, ldg=0, scale=1.0, pre=1, qw=NULL, qb=NULL, eps=1e-6,
            st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(r=NULL), ARG), (dict(ro=NULL, x=NULL), ARG), (dict(rt=0), ARG), (dict(yt=4), ARG), (dict(xt=0), ARG),
    (dict(post=3), ARG), (dict(pre=-1), ARG), (dict(gate=GOOD, gt=7), ARG), (dict(eps=-1e-6), ARG),
    (dict(eps=float("nan")), ARG), (dict(ldro=256), ARG), (dict(x=GOOD), ARG), (dict(x=OTHER), ARG),
    (dict(ro=GOOD), ARG),
    (dict(m=0), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=(1 << 22) + 1), SHAPE),
    (dict(ldy=127), SHAPE), (dict(ldr=127), SHAPE), (dict(ldx=0), SHAPE), (dict(ro=P(0x50000), ldro=1), SHAPE),
    (dict(gate=GOOD, gt=F32, ldg=127), SHAPE), (dict(ldy=1 << 62), SHAPE),
    (dict(y=P(0x10002)), ALIGN), (dict(x=P(0x30001)), ALIGN), (dict(pw=P(0x10002)), ALIGN),
    (dict(gate=P(0x10001), gt=BF16), ALIGN),
])
def test_norm_refusals(lib, over, status):
    assert lib.lowbit_norm_residual(*{**NORM, **over}.values()) == status


LOGITS = dict(y=GOOD, yt=F32, ldy=100, n=100, b=2, tok=GOOD, tcap=10, ldt=10, pl=NULL, tl=NULL, rep=NULL, freq=NULL,
              pres=NULL, bi=GOOD, bv=GOOD, bcap=4, ldb=4, bl=NULL, mask=GOOD, rows=2, ldm=4, mr=NULL, out=OTHER,
              ldo=100, idx=THIRD, val=THIRD, ws=GOOD, wsb=1 << 20, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(y=NULL), ARG), (dict(yt=5), ARG), (dict(out=NULL, idx=NULL, val=NULL), ARG), (dict(idx=NULL), ARG),
    (dict(bv=NULL), ARG), (dict(bi=NULL), ARG), (dict(out=GOOD, yt=BF16), ARG), (dict(out=GOOD, ldo=200), ARG),
    (dict(n=0), SHAPE), (dict(n=1 << 31), SHAPE), (dict(b=0), SHAPE), (dict(b=65536), SHAPE), (dict(ldy=99), SHAPE),
    (dict(ldo=99), SHAPE), (dict(tcap=-1), SHAPE), (dict(ldt=9), SHAPE), (dict(tcap=1 << 30, ldt=1 << 30), SHAPE),
    (dict(ldb=3), SHAPE), (dict(bcap=-2), SHAPE), (dict(bcap=16385, ldb=16385), SHAPE), (dict(ldm=3), SHAPE),
    (dict(rows=0), SHAPE),
    # n * b of 2^35 passes (the address is then refused), more does not
    (dict(n=1 << 20, b=1 << 15, ldy=1 << 20, ldo=1 << 20, ldm=1 << 15, rows=1 << 15, idx=NULL, val=NULL,
          y=P(0x10002)), ALIGN),
    (dict(n=(1 << 20) + 1, b=1 << 15, ldy=1 << 21, ldo=1 << 21), SHAPE),
    (dict(y=P(0x10002)), ALIGN), (dict(tok=P(0x10002)), ALIGN), (dict(mask=P(0x10001)), ALIGN),
    (dict(ws=NULL), WS), (dict(wsb=8), WS), (dict(ws=P(0x10008)), ALIGN),
])
def test_logits_refusals(lib, over, status):
    assert lib.lowbit_logits_process(*{**LOGITS, **over}.values()) == status


LORA = dict(x=GOOD, xt=F16, ldx=128, ids=GOOD, m=2, n=100, k=128, r=16, slots=4, a=GOOD, b=GOOD, ranks=NULL,
            scales=NULL, y=OTHER, yt=F32, ldy=100, ws=GOOD, wsb=1 << 26, st=NULL)


@pytest.mark.parametrize("over,status", [
    (dict(x=NULL), ARG), (dict(ids=NULL), ARG), (dict(a=NULL), ARG), (dict(b=NULL), ARG), (dict(y=NULL), ARG),
    (dict(xt=F32), ARG), (dict(yt=F16), ARG), (dict(yt=BF16), ARG),
    (dict(m=0), SHAPE), (dict(n=0), SHAPE), (dict(n=1 << 31), SHAPE), (dict(k=0), SHAPE), (dict(k=100), SHAPE),
    (dict(r=0), SHAPE), (dict(r=12), SHAPE), (dict(r=264), SHAPE), (dict(slots=0), SHAPE), (dict(slots=4097), SHAPE),
    (dict(ldx=120), SHAPE), (dict(ldy=99), SHAPE),
    (dict(ldx=132), ALIGN), (dict(x=P(0x10008)), ALIGN), (dict(a=P(0x10008)), ALIGN), (dict(b=P(0x10002)), ALIGN),
    (dict(y=P(0x20002)), ALIGN), (dict(ids=P(0x10002)), ALIGN), (dict(ws=P(0x10008)), ALIGN),
    (dict(ws=NULL), WS), (dict(wsb=16), WS),
])
def test_lora_refusals(lib, over, status):
    assert lib.lowbit_lora_accumulate(*{**LORA, **over}.values()) == status


def test_workspace_queries(lib):
    for n, b in ((1, 1), (151936, 64), (32003, 33)):
        assert lowbit.lowbit_logits_workspace_bytes(n, b) > 0
    assert lowbit.lowbit_logits_workspace_bytes(0, 1) == 0 == lowbit.lowbit_logits_workspace_bytes(10, 0)
    for args in ((1, 1, 8, 8, 1), (8, 34816, 5120, 64, 16), (4096, 17408, 5120, 32, 8)):
        m, n, k, r, slots = args
        assert lowbit.lowbit_lora_workspace_bytes(*args) >= m * r * 4  # the inner values of every row
    assert lowbit.lowbit_lora_workspace_bytes(8, 100, 128, 12, 4) == 0
    assert lowbit.lowbit_lora_workspace_bytes(0, 100, 128, 16, 4) == 0


def test_binding_rejects_host_tensors_and_wrong_types():
    import torch

    x = torch.zeros(2, 128, dtype=torch.float16)
    with pytest.raises(TypeError):
        lowbit.lowbit_norm_residual(None, x, pre="rms")
    with pytest.raises(TypeError):
        lowbit.lowbit_norm_residual(None, torch.zeros(2, 128, dtype=torch.int32), pre="rms")
    with pytest.raises(TypeError):
        lowbit.lowbit_logits_process(torch.zeros(2, 100))
    with pytest.raises(TypeError, match="not list"):
        lowbit.lowbit_logits_process([1.0, 2.0])
    with pytest.raises(TypeError):
        lowbit.lowbit_lora_accumulate(x, torch.zeros(2, dtype=torch.int32), torch.zeros(1, 8, 128), torch.zeros(1, 4, 8),
                                      torch.zeros(2, 4))


def test_argument_module_counts_its_arguments():
    from bit_matmul_lowbit_amd import _marshal

    for f in (_marshal.bind, _marshal.norm, _marshal.logits, _marshal.lora):
        with pytest.raises(TypeError, match="expected"):
            f("name")


@pytest.mark.parametrize("call", [
    lambda t: lowbit.lowbit_norm_residual(None, t(2, 8), pre="rms"),
    lambda t: lowbit.lowbit_norm_residual(None, 3),
    lambda t: lowbit.lowbit_norm_residual(None, t(2, 8), pre="rms", x_dtype="float16"),
    lambda t: lowbit.lowbit_norm_residual(None, t(2, 8), scale="a"),
    lambda t: lowbit.lowbit_logits_process(t(100)),
    lambda t: lowbit.lowbit_logits_process([1.0]),
    lambda t: lowbit.lowbit_lora_accumulate(t(1, 8), t(1), t(1, 8, 8), t(1, 8, 8), t(1, 8)),
])
def test_the_binding_refuses_host_tensors_and_other_objects(call):
    import torch

    with pytest.raises(TypeError):
        call(torch.zeros)
