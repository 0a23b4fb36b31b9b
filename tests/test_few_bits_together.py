"""The residual stream's and the few-bit calls as programs make them: at once, on one matrix twice, captured as the first
calls of a process, and at the ends of the range."""
import os
import subprocess
import sys

import pytest
import torch

from tests.conftest import ROOT
from tests.test_mx import BF, F32, buffers, check_product, quantised, rng_of, ss  # noqa: F401

gpu = pytest.mark.gpu


@gpu
def test_products_on_two_streams(ss):  # noqa: F811
    """Large and few-row products, and a loss, side by side give what they give alone."""
    gen = torch.Generator("cuda").manual_seed(1)
    jobs = []
    for M, N, K, format in ((2500, 2600, 300, 0), (3, 2048, 4096, 0), (300, 900, 520, 1), (2048, 5632, 256, 1), (60, 700, 2048, 1),
                            (30, 1500, 1001, 0)):
        (qa, _), (qb, _) = quantised(ss, M, K, format, gen), quantised(ss, N, K, format, gen)
        jobs.append((qa, qb, K, format, *(torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2))))
    h, w = (torch.randn(n, 512, generator=gen, device="cuda").to(BF) for n in (300, 8000))
    y = torch.randint(0, 8000, (300,), generator=gen, device="cuda")
    want, loss = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(ss.ss_linear_ce_workspace(300, 512, 8000, False), dtype=torch.uint8, device="cuda")
    for qa, qb, K, format, alone, _ in jobs:
        ss.ss_mx_matmul(*qa, *qb, K, format, alone)
    ss.ss_linear_cross_entropy(h, w, y, want, ws)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for r in range(6):
        for i, (qa, qb, K, format, _, out) in enumerate(jobs):
            ss.ss_mx_matmul(*qa, *qb, K, format, out, stream=streams[i % 2])
        ss.ss_linear_cross_entropy(h, w, y, loss, ws, stream=streams[2])
    torch.cuda.synchronize()
    for *_, alone, out in jobs:
        assert torch.equal(out, alone)
    assert torch.equal(loss, want)


@gpu
@pytest.mark.parametrize("format", [0, 1])
@pytest.mark.parametrize("n,K", [(40, 300), (700, 129), (2600, 200)])
def test_product_of_a_matrix_with_itself(ss, n, K, format):  # noqa: F811
    q, a = quantised(ss, n, K, format, torch.Generator("cuda").manual_seed(n))
    out = torch.empty(n, n, device="cuda")
    ss.ss_mx_matmul(*q, *q, K, format, out)
    check_product(out, a, a)


@gpu
@pytest.mark.parametrize("format", [0, 1])
def test_captured_training_products(ss, format):  # noqa: F811
    """A captured projection and its gradients round anew once the offset on the device is another."""
    T, K, N = 200, 328, 456
    gen = torch.Generator("cuda").manual_seed(2)
    x, w, dy = (torch.randn(r, c, generator=gen, device="cuda").to(BF) for r, c in ((T, K), (N, K), (T, N)))
    rng = rng_of(3, 0)
    q = {name: buffers(ss, r, c, format) for name, r, c in (("x", T, K), ("xt", K, T), ("w", N, K), ("wt", K, N), ("d", T, N), ("dt", N, T))}
    y, dx, dw = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty_like(x), torch.empty_like(w)

    def step():
        ss.ss_mx_quantize(x, format, *q["x"], *q["xt"])
        ss.ss_mx_quantize(w, format, *q["w"], *q["wt"])
        ss.ss_mx_matmul(*q["x"], *q["w"], K, format, y)
        ss.ss_mx_quantize(dy, format, *q["d"], *q["dt"], rng=rng)
        ss.ss_mx_matmul(*q["d"], *q["wt"], N, format, dx)
        ss.ss_mx_matmul(*q["dt"], *q["xt"], T, format, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for offset in (1, 2):
        rng[1] = offset
        graph.replay()
        got = [t.clone() for t in (y, dx, dw)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw)))
        seen.append(got)
    assert torch.equal(seen[0][0], seen[1][0]) and not torch.equal(seen[0][1], seen[1][1])


FIRST = """
import torch, sharded_state_gb300 as ss
x, r = (torch.randn(300, 1000, device="cuda").to(torch.bfloat16) for _ in range(2))
w, up = torch.ones(1000, dtype=torch.bfloat16, device="cuda"), torch.randn(700, 1000, device="cuda").to(torch.bfloat16)
rng = torch.tensor([1, 2], device="cuda")
u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
q, k = ([u8(n) for n in ss.ss_mx_bytes(rows, 1000, 1)] for rows in (300, 700))
outs = [torch.zeros_like(x) for _ in range(4)] + [torch.zeros(300, device="cuda"), torch.zeros_like(w),
                                                 torch.zeros(300, 700, device="cuda")]
h, y, dh, dx, rstd, dw, z = outs
ws = u8(ss.ss_rms_norm_workspace(300, 1000))
def step():
    ss.ss_rms_norm(x, w, 1e-5, out=y, residual=r, sum_out=h, rstd_out=rstd, mx_data=q[0], mx_scales=q[1], dropout=0.1, rng=rng)
    ss.ss_mx_quantize(up, 1, *k)
    ss.ss_mx_matmul(*q, *k, 1000, 1, z)
    ss.ss_rms_norm_backward(y, h, w, rstd, dh, ws, d_x=dx, d_weight=dw, dropout=0.1, rng=rng)
    ss.ss_dropout(dx, dx, 0.5, rng)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
got = [t.clone() for t in outs]
assert all(bool((t != 0).any()) for t in got)
for t in outs: t.zero_()
step()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
print("equal")
"""


@gpu
def test_captured_as_the_first_calls(ss):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=ROOT), cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stderr[-2000:]


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_up_to_the_largest_sum_of_squares(ss, dtype):  # noqa: F811
    """A row's sum of squares may be any fp32 number: 4096 elements of 2^57 sum up to 2^126, of 2^58 beyond the largest."""
    x = torch.ones(4, 4096, dtype=dtype, device="cuda")
    x[0] *= 2.0 ** 57
    x[1] *= 2.0 ** 58
    x[2] *= 2.0 ** -62
    x[3] = 0
    w, out, rstd = torch.ones(4096, dtype=dtype, device="cuda"), torch.empty_like(x), torch.empty(4, device="cuda")
    ss.ss_rms_norm(x, w, 0.0, out=out, rstd_out=rstd)
    assert out[:3, 0].tolist() == [1.0, 0.0, 1.0] and rstd[:3].tolist() == [2.0 ** -57, 0.0, 2.0 ** 62]
    assert torch.equal(out[:3], out[:3, :1].expand(3, 4096)) and bool(out[3].isnan().all())
    ss.ss_rms_norm(x, w, 1e-6, out=out, rstd_out=rstd)
    assert bool((out[3] == 0).all())
