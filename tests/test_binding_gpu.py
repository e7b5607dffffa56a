"""What the binding of the operators beside the products refuses before the
library is called: other types, shapes, strides, devices and sizes."""
import pytest

from bit_matmul_lowbit_amd import lowbit

pytestmark = pytest.mark.gpu


def _f(*shape, dtype="float32"):
    import torch

    return torch.zeros(shape, dtype=getattr(torch, dtype), device="cuda")


def _norm(**over):
    args = dict(y=_f(4, 256), r=_f(4, 256), post="rms", post_w=_f(256), pre="rms", pre_w=_f(256))
    args.update(over)
    return lowbit.lowbit_norm_residual(**args)


def _logits(**over):
    i32 = "int32"
    args = dict(y=_f(3, 1000), tokens=_f(3, 10, dtype=i32), prompt_len=_f(3, dtype=i32), total_len=_f(3, dtype=i32),
                repetition=_f(3) + 1, bias_ids=_f(3, 4, dtype=i32), bias_vals=_f(3, 4), mask=_f(3, 32, dtype=i32))
    args.update(over)
    return lowbit.lowbit_logits_process(**args)


def _lora(**over):
    args = dict(x=_f(5, 128, dtype="float16"), ids=_f(5, dtype="int32"), a=_f(2, 8, 128, dtype="float16"),
                b=_f(2, 40, 8, dtype="float16"), y=_f(5, 40), ranks=_f(2, dtype="int32"), scales=_f(2))
    args.update(over)
    return lowbit.lowbit_lora_accumulate(**args)


def test_the_plain_calls_pass():
    import torch

    _norm()
    _logits()
    _lora()
    torch.cuda.synchronize()


@pytest.mark.parametrize("call,over,error", [
    (_norm, lambda: dict(r=_f(4, 255)), ValueError),
    (_norm, lambda: dict(r=_f(2, 2, 256)), ValueError),
    (_norm, lambda: dict(y=_f(256, 4).t()), ValueError),
    (_norm, lambda: dict(y=_f(4, 256, dtype="int32")), TypeError),
    (_norm, lambda: dict(y=_f(4, 256).cpu()), TypeError),
    (_norm, lambda: dict(post="max"), KeyError),
    (_norm, lambda: dict(post_w=_f(255)), ValueError),
    (_norm, lambda: dict(post_w=_f(512)[::2]), ValueError),
    (_norm, lambda: dict(post_w=_f(256, dtype="float16")), TypeError),
    (_norm, lambda: dict(gate=_f(255)), ValueError),
    (_norm, lambda: dict(gate=_f(3, 256)), ValueError),
    (_norm, lambda: dict(r_out=_f(4, 256, dtype="float16")), TypeError),
    (_norm, lambda: dict(y=None, r_out=_f(4, 256)), ValueError),
    (_norm, lambda: dict(pre=None, x_out=_f(4, 256)), ValueError),
    (_norm, lambda: dict(r=_f(1, 256).expand(4, 256)), lowbit.LowbitError),
    (_norm, lambda: dict(eps=-1.0), lowbit.LowbitError),
    (_logits, lambda: dict(y=_f(3, 1000, dtype="int32")), TypeError),
    (_logits, lambda: dict(tokens=_f(2, 10, dtype="int32")), ValueError),
    (_logits, lambda: dict(tokens=_f(30, dtype="int32")), ValueError),
    (_logits, lambda: dict(tokens=_f(3, 10, dtype="int64")), TypeError),
    (_logits, lambda: dict(tokens=_f(3, 20, dtype="int32")[:, ::2]), ValueError),
    (_logits, lambda: dict(total_len=_f(2, dtype="int32")), ValueError),
    (_logits, lambda: dict(bias_vals=None), ValueError),
    (_logits, lambda: dict(bias_vals=_f(3, 5)), ValueError),
    (_logits, lambda: dict(mask=_f(3, 31, dtype="int32")), ValueError),
    (_logits, lambda: dict(mask=_f(2, 32, dtype="int32")), ValueError),
    (_logits, lambda: dict(out=_f(3, 1000, dtype="float16")), TypeError),
    (_logits, lambda: dict(out=_f(3, 999)), ValueError),
    (_logits, lambda: dict(top1=False), lowbit.LowbitError),
    (_logits, lambda: dict(top1=False, idx=_f(3, dtype="int32")), ValueError),
    (_logits, lambda: dict(idx=_f(2, dtype="int32")), ValueError),
    (_logits, lambda: dict(workspace=_f(8, dtype="uint8")), lowbit.LowbitError),
    (_lora, lambda: dict(x=_f(5, 120, dtype="float16")), ValueError),
    (_lora, lambda: dict(x=_f(5, 128)), (TypeError, lowbit.LowbitError)),
    (_lora, lambda: dict(ids=_f(4, dtype="int32")), ValueError),
    (_lora, lambda: dict(ids=_f(5, dtype="int64")), TypeError),
    (_lora, lambda: dict(a=_f(2, 8, 128, dtype="bfloat16")), TypeError),
    (_lora, lambda: dict(a=_f(3, 8, 128, dtype="float16")), ValueError),
    (_lora, lambda: dict(b=_f(2, 40, 16, dtype="float16")), ValueError),
    (_lora, lambda: dict(y=_f(5, 41)), ValueError),
    (_lora, lambda: dict(y=_f(4, 40)), ValueError),
    (_lora, lambda: dict(y=_f(5, 40, dtype="float16")), lowbit.LowbitError),
    (_lora, lambda: dict(scales=_f(1)), ValueError),
    (_lora, lambda: dict(workspace=_f(8, dtype="uint8")), lowbit.LowbitError),
    (_lora, lambda: dict(x=_f(5, 132, dtype="float16")[:, 4:]), lowbit.LowbitError),
])
def test_refusals(call, over, error):
    with pytest.raises(error):
        call(**over())


class _OtherDevice:
    device_index = 1
    cuda_stream = 0


@pytest.mark.parametrize("call", [_norm, _logits, _lora])
def test_a_stream_of_another_device_is_refused(call):
    with pytest.raises(ValueError):
        call(stream=_OtherDevice())


@pytest.mark.parametrize("op", ["norm", "logits"])
def test_outputs_on_another_stream_do_not_reuse_its_memory(op):
    """What the current stream freed may still be written by work that waits
    there: a call on another stream gets other memory for its outputs."""
    import torch

    side = torch.cuda.Stream()
    r, y = _f(4, 200000), _f(70000, 64)
    torch.cuda.synchronize()

    def run():
        if op == "norm":
            return lowbit.lowbit_norm_residual(None, r, pre="rms", x_dtype=torch.float32, stream=side)[1:]
        return lowbit.lowbit_logits_process(y[:60000], stream=side)[1:]

    sizes = [t.numel() for t in run()]
    torch.cuda.synchronize()
    freed = [torch.empty(n, dtype=torch.float32, device="cuda") for n in sizes]
    held = {t.data_ptr() for t in freed}
    del freed
    outs = run()
    torch.cuda.synchronize()
    assert not held & {t.data_ptr() for t in outs}
