"""What random rounding gives on average: the input up to the format's largest element, that element beyond it."""
import pytest
import torch

from tests import stream_reference as ref
from tests.test_mx import BF, buffers, rng_of, ss  # noqa: F401

# (inputs in units of the scale, up to their block's largest), and the steps around them
INPUTS = {0: ([7.5, 5.25, 4.5, 6.0, 2.3125, 0.203125, 6.5], [None, 2.0, 2.0, 0.0, 1.0, 0.5, None]),
          1: ([508.0, 440.0, 448.0, 100.5, 0.0009765625, 450.0], [None, 32.0, 0.0, 8.0, 2.0 ** -9, None])}


def check(out, format):
    values, steps = INPUTS[format]
    most = ref.table(format)[-1]
    for i, (x, step) in enumerate(zip(values, steps)):
        got = out[:, i].double()
        if step is None:  # beyond the largest element: cut to it every time
            assert x > most and bool((got == most).all())
        elif step == 0:
            assert bool((got == x).all())
        else:  # a rounding is off by less than a step: six standard deviations, half a step / 64 each, and 2^-16 of it
            assert abs(float(got.mean()) - x) <= 6 * step / 128 + 2.0 ** -16 * step, (x, float(got.mean()))
            assert len(got.unique()) == 2


def rows_of(format):
    x = torch.zeros(4096, 32)
    x[:, :len(INPUTS[format][0])] = torch.tensor(INPUTS[format][0])
    assert torch.equal(x.to(BF).float(), x)
    return x.to(BF)


@pytest.mark.parametrize("format", [0, 1])
def test_the_plain_form(format):
    x = rows_of(format)
    check(ref.quantise(x, format, ref.bits16(12345, 77, *x.shape))[3], format)


@pytest.mark.gpu
@pytest.mark.parametrize("format", [0, 1])
def test_the_kernel(ss, format):  # noqa: F811
    x = rows_of(format).cuda()
    q, out = buffers(ss, 4096, 32, format), torch.empty(4096, 32, device="cuda")
    ss.ss_mx_quantize(x, format, *q, rng=rng_of())
    ss.ss_mx_dequantize(*q, format, out)
    check(out.cpu(), format)
    want = ref.quantise(x, format, ref.bits16(12345, 77, 4096, 32))[3]
    assert torch.equal(out.cpu().double(), want)
