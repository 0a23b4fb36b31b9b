"""README's training example along the residual stream: what it shows can be done for one layer after another."""
import os
import re

import pytest
import torch

from tests.conftest import ROOT
from tests.stream_reference import keep_mask
from tests.test_norm import dropped, rng_of, ss  # noqa: F401


def example():
    """The lines of the example, as README has them."""
    text = open(os.path.join(ROOT, "README.md")).read()
    at = text.index("A layer's step along the residual stream")
    return "\n".join(line[4:] for line in re.match(r"[^\n]*\n\n((?:    [^\n]*\n)+)", text[at:]).group(1).splitlines())


class Names(dict):
    """Every name stands for itself."""

    def __missing__(self, key):
        return key


class Calls:
    def __init__(self):
        self.made = {}

    def __getattr__(self, name):
        return lambda *args, **kw: self.made.setdefault(name, []).append((args, kw))


def test_example_keeps_what_its_backward_pass_reads():
    calls = Calls()
    exec(example(), {}, Names(ss=calls, torch=Calls()))
    (_, forward), (back, _) = calls.made["ss_rms_norm"][0], calls.made["ss_rms_norm_backward"][0]
    h, rstd = back[1], back[3]
    assert forward["sum_out"] == h and forward["rstd_out"] == rstd
    # the stream over its own input would be the next layer's h by the time the backward pass comes here
    assert h != forward["residual"]
    assert len(calls.made["ss_mx_quantize"]) == 2 and len(calls.made["ss_mx_matmul"]) == 2


@pytest.mark.gpu
def test_two_layers_with_a_sum_each(ss):  # noqa: F811
    """The example's calls for two layers, against autograd in 64 bits.  A call is off by less than 100 * 2^-24 of its
    result's norm; in four that follow one another, each with a derivative of norm below 1 / (1 - d) * max w * rstd < 3,
    that is below 4 * 100 * 2^-24 * 3^3 < 1e-3 of the gradients'."""
    rows, cols, p = 70, 264, 0.1
    gen = torch.Generator("cuda").manual_seed(4)
    x, stream, d_y, d_stream = (torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(4))
    weight = [1 + 0.2 * torch.randn(cols, generator=gen, device="cuda") for _ in range(2)]
    rngs = [rng_of(5, layer) for layer in range(2)]
    h, y, dx, dh = ([torch.empty_like(x) for _ in range(2)] for _ in range(4))
    rstd, dw = [torch.empty(rows, device="cuda") for _ in range(2)], [torch.empty(cols, device="cuda") for _ in range(2)]
    ws = torch.empty(ss.ss_rms_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    for i in range(2):  # the second layer's branch is the first one's norm
        ss.ss_rms_norm(y[0] if i else x, weight[i], 1e-5, out=y[i], residual=h[0] if i else stream, sum_out=h[i],
                       rstd_out=rstd[i], dropout=p, rng=rngs[i])
    for i in (1, 0):
        ss.ss_rms_norm_backward(dx[1] if i == 0 else d_y, h[i], weight[i], rstd[i], dh[i], ws,
                                d_sum=dh[1] if i == 0 else d_stream, d_x=dx[i], d_weight=dw[i], dropout=p, rng=rngs[i])
    leaves = [t.double().requires_grad_() for t in (x, stream, *weight)]
    branch, s = leaves[0], leaves[1]
    for i in range(2):
        s = dropped(branch, keep_mask(rngs[i], rows, cols, p), p) + s
        branch = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-5) * leaves[2 + i]
    want = torch.autograd.grad((branch * d_y.double()).sum() + (s * d_stream.double()).sum(), leaves)
    for got, ref in zip((dx[0], dh[0], *dw), want):
        assert float((got.double() - ref).norm()) <= 1e-3 * float(ref.norm())
