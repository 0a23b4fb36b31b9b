"""Microscaled floats -- quantisation, back, products -- against plain forms in 64 bits.

Quantisation is exact but for its one rounding, so codes and scales have to be equal.  A product is a sum of K exact
products in the tensor cores' fp32 accumulator, 64 (MXFP4) or 32 (MXFP8) an instruction, and over up to 8 shares of k:
its error is at most (K / 32 + 10) * 2^-22 * sum_k |a_k b_k| (2^-22: an add that keeps 24 bits and may truncate, twice
over for the products' own alignment), and half a step of the result's type.
"""
import math

import pytest
import torch

from tests import stream_reference as ref
from tests.test_norm import block, matrix, outside_kept, randn, rng_of

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMATS = [0, 1]


@pytest.fixture(scope="module")
def ss():
    import __graft_entry__
    __graft_entry__.build()
    import sharded_state_gb300 as ss
    return ss


def buffers(ss, rows, cols, format, fill=0xFF):
    """Buffers of a quantised matrix (0xFF: NaN scales wherever nothing is written), 32 bytes longer."""
    return [torch.full((n + 32,), fill, dtype=torch.uint8, device="cuda") for n in ss.ss_mx_bytes(rows, cols, format)]


def check_buffers(ss, q, x, format, bits=None):
    rows, cols = x.shape
    code, sign, byte = ref.unpack(*q, rows, cols, format)
    want_code, want_sign, want_byte, _ = ref.quantise(x, format, bits)
    blocks = want_byte.shape[1]
    assert torch.equal(byte[:, :blocks], want_byte)
    assert bool((byte[:, blocks:] == 0).all()) and bool((code[:, cols:] == 0).all())
    assert torch.equal(code[:, :cols], want_code)
    live = want_code != 0  # the sign of a zero is not looked at
    assert torch.equal(sign[:, :cols][live], want_sign[live])
    for t, n in zip(q, ss.ss_mx_bytes(rows, cols, format)):
        assert bool((t[n:] == 0xFF).all())


# ---------------------------------------------------------------------------
# on the CPU
# ---------------------------------------------------------------------------

def test_sizes(ss):
    assert ss.ss_mx_bytes(1, 1, ss.SS_MXFP4) == (64, 512)
    assert ss.ss_mx_bytes(129, 257, ss.SS_MXFP8) == (129 * 384, 2 * 3 * 512)
    assert ss.ss_mx_bytes(0, 5, 0) == (0, 0) and ss.ss_mx_bytes((1 << 31) - 1, (1 << 31) - 1, 1)[0] > 1 << 61
    for bad in ((-1, 1, 0), (1, -1, 0), (1, 1, 2), (1 << 31, 1, 0)):
        with pytest.raises(ss.ShardStateError):
            ss.ss_mx_bytes(*bad)


def test_refusals_of_the_c_calls(ss):
    lib, n, a = ss.lib(), ss.ss_launch_count(), 4096

    def quant(**kw):
        s = dict(rows=4, cols=8, elem_bytes=2, x=a, stride=8, format=0, data=a, scales=a, t_data=a, t_scales=a, rng=a)
        return lib.ss_mx_quantize(block(ss._MX_QUANT, s, kw), None)
    assert quant(rows=-1) == quant(cols=-1) == quant(elem_bytes=1) == quant(format=2) == quant(x=None) == ss.SS_EINVAL
    assert quant(data=None) == quant(scales=None) == quant(t_data=None) == quant(t_scales=None) == ss.SS_EINVAL
    none = dict(data=None, scales=None, t_data=None, t_scales=None)
    assert quant(**none) == quant(stride=7) == ss.SS_EINVAL
    assert quant(x=a + 1) == quant(data=a + 8) == quant(scales=a + 4) == quant(t_data=a + 8) == ss.SS_EALIGN
    assert quant(t_scales=a + 8) == quant(rng=a + 4) == quant(elem_bytes=4, x=a + 2) == ss.SS_EALIGN
    assert quant(rows=1 << 31) == quant(stride=1 << 60) == ss.SS_EOVERFLOW
    assert quant(rows=(1 << 31) - 1, cols=(1 << 31) - 1, stride=1 << 31) == ss.SS_EOVERFLOW
    assert quant(rows=0, **none) == quant(cols=0) == ss.SS_OK and lib.ss_mx_quantize(None, None) == ss.SS_EINVAL

    def back(rows=4, cols=8, format=1, data=a, scales=a, out=a, stride=8, eb=4):
        return lib.ss_mx_dequantize(rows, cols, format, data, scales, out, stride, eb, None)
    assert back(rows=-1) == back(format=-1) == back(data=None) == back(scales=None) == back(out=None) == ss.SS_EINVAL
    assert back(stride=7) == back(eb=3) == ss.SS_EINVAL
    assert back(data=a + 8) == back(scales=a + 8) == back(out=a + 2) == ss.SS_EALIGN
    assert back(cols=1 << 31, stride=1 << 31) == back(stride=1 << 62) == ss.SS_EOVERFLOW
    assert back(rows=0) == ss.SS_OK

    def product(**kw):
        s = dict(M=4, N=8, K=32, format=0, a_data=a, a_scales=a, b_data=a, b_scales=a, out=a, out_stride=8, elem_bytes=2)
        return lib.ss_mx_matmul(block(ss._MX_PRODUCT, s, kw), None)
    assert product(M=-1) == product(N=-1) == product(K=0) == product(format=5) == product(elem_bytes=8) == ss.SS_EINVAL
    for field in ("a_data", "a_scales", "b_data", "b_scales", "out"):
        assert product(**{field: None}) == ss.SS_EINVAL and product(**{field: a + 1}) == ss.SS_EALIGN, field
    assert product(out_stride=7) == ss.SS_EINVAL and product(K=1 << 31) == product(out_stride=1 << 62) == ss.SS_EOVERFLOW
    assert product(M=0) == product(N=0) == ss.SS_OK and lib.ss_mx_matmul(None, None) == ss.SS_EINVAL
    assert ss.ss_launch_count() == n


def test_the_plain_form_on_known_values():
    """The formats' specification by hand: ties to even, saturation, the lowest scale."""
    x = torch.tensor([[4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -7.9, -0.0, 0.26]])
    _, _, byte, v = ref.quantise(x, 0)
    assert byte.tolist() == [[127]]
    assert v.tolist() == [[4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, -6.0, 0.0, 0.5]]
    _, _, byte, v = ref.quantise(torch.tensor([[500.0, 17.0, 2.0 ** -10, 1.5 * 2.0 ** -9]]), 1)
    assert byte.tolist() == [[127]] and v.tolist() == [[448.0, 16.0, 0.0, 2.0 ** -8]]
    assert ref.quantise(torch.zeros(1, 5), 0)[2].tolist() == [[0]]


# ---------------------------------------------------------------------------
# quantisation and back
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,extra,offset,random", [
    (1, 1, 0, 0, False), (1, 4096, 0, 0, False), (3, 33, 0, 0, True), (128, 128, 0, 0, True), (129, 257, 0, 1, False),
    (50, 64, 8, 0, False), (300, 1001, 0, 0, True), (1021, 200, 3, 5, True), (31, 8, 0, 0, True)])
def test_quantise(ss, format, dtype, rows, cols, extra, offset, random):
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    x = randn(rows, cols, dtype, gen, extra=extra, offset=offset)
    x *= torch.exp2(8 * torch.randn(rows, cols, generator=gen, device="cuda")).to(dtype)
    rng = rng_of(99, -7) if random else None
    bits = ref.bits16(99, -7, rows, cols) if random else None
    q, t = buffers(ss, rows, cols, format), buffers(ss, cols, rows, format)
    ss.ss_mx_quantize(x, format, *q, *t, rng=rng)
    check_buffers(ss, q, x, format, bits)
    check_buffers(ss, t, x.t(), format, bits.t() if random else None)
    for which in ("rows", "columns"):  # either alone gives the same bits
        q1, t1 = buffers(ss, rows, cols, format), buffers(ss, cols, rows, format)
        ss.ss_mx_quantize(x, format, *(q1 if which == "rows" else (None, None)),
                          *(t1 if which == "columns" else (None, None)), rng=rng)
        for a, b in zip(q1, q) if which == "rows" else zip(t1, t):
            assert torch.equal(a, b)
    for out_dtype in (BF, F32):
        out, buf = matrix(rows, cols, out_dtype, extra, offset, fill=5.0)
        ss.ss_mx_dequantize(*q, format, out)
        want = ref.values(*q, rows, cols, format)
        assert torch.equal(out.cpu(), want.to(out_dtype)) and outside_kept(buf, out, 5.0)


@gpu
@pytest.mark.parametrize("format", FORMATS)
def test_every_element_and_tie(ss, format):
    """Every listed magnitude, every middle between two, and their neighbours in fp32, at scales from the lowest to the
    highest; and all bf16 numbers."""
    t = ref.table(format).float()
    v = torch.cat([t, (t[1:] + t[:-1]) / 2])
    v = torch.cat([v, torch.nextafter(v, torch.tensor(0.0)), torch.nextafter(v, torch.tensor(1e9))])
    v = torch.cat([v, -v])
    top = float(2 ** (2 if format == 0 else 8))
    v = v[v.abs() < 2 * top]
    pad = -len(v) % 31
    v = torch.cat([v, torch.zeros(pad)]).view(-1, 31)
    rows = [torch.cat([torch.full((v.shape[0], 1), top), v], 1) * 2.0 ** e for e in (-127, -126, -20, 0, 60, 119)]
    x = torch.cat(rows).view(1, -1).cuda()
    q = buffers(ss, 1, x.shape[1], format)
    ss.ss_mx_quantize(x, format, *q)
    check_buffers(ss, q, x, format)
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF).view(256, 256).cuda()
    q, tq = buffers(ss, 256, 256, format), buffers(ss, 256, 256, format)
    ss.ss_mx_quantize(every, format, *q, *tq)
    check_buffers(ss, q, every, format)
    check_buffers(ss, tq, every.t(), format)


@gpu
@pytest.mark.parametrize("format", FORMATS)
def test_blocks_with_special_values(ss, format):
    x = torch.ones(64, 128, device="cuda")
    x[0, 5], x[1, 40], x[2, 127], x[3], x[4, 64:96] = math.nan, math.inf, -math.inf, 0.0, 1e-42
    x[5, 0] = torch.finfo(F32).max
    q, t = buffers(ss, 64, 128, format), buffers(ss, 128, 64, format)
    ss.ss_mx_quantize(x, format, *q, *t, rng=rng_of())
    bits = ref.bits16(12345, 77, 64, 128)
    check_buffers(ss, q, x, format, bits)
    check_buffers(ss, t, x.t(), format, bits.t())
    out = torch.empty(64, 128, device="cuda")
    ss.ss_mx_dequantize(*q, format, out)
    bad = torch.zeros(64, 128, dtype=torch.bool, device="cuda")
    bad[0, :32] = bad[1, 32:64] = bad[2, 96:] = True
    assert torch.equal(torch.isnan(out), bad)


@gpu
@pytest.mark.parametrize("format", FORMATS)
def test_stochastic_rounding_is_even_handed(ss, format):
    """The mean of 4096 roundings of one number: each is off by less than a step, so the mean's standard deviation is
    below half a step / 64; six of them."""
    x = torch.full((4096, 32), 1.0, device="cuda")
    x[:, 0], x[:, 1] = (4.0, 2.3) if format == 0 else (256.0, 100.7)
    step = 1.0 if format == 0 else 8.0
    q = buffers(ss, 4096, 32, format)
    ss.ss_mx_quantize(x, format, *q, rng=rng_of())
    out = torch.empty_like(x)
    ss.ss_mx_dequantize(*q, format, out)
    assert abs(float(out[:, 1].mean()) - float(x[0, 1])) <= 6 * step / 128 + 2.0 ** -16 * step
    assert bool((out[:, 2:] == 1).all())


@gpu
def test_quantise_offsets_past_32_bits(ss):
    """Rows more than 2^32 bytes apart in x and in out, and a quantised matrix of more than 2^31 bytes."""
    stride = (1 << 31) + 24
    buf = torch.zeros(2 * stride + 512, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (3, 300), (stride, 1))
    x.copy_(torch.randn(3, 300, device="cuda"))
    q, t = buffers(ss, 3, 300, 0), buffers(ss, 300, 3, 0)
    ss.ss_mx_quantize(x, 0, *q, *t)
    check_buffers(ss, q, x, 0)
    check_buffers(ss, t, x.t(), 0)
    ss.ss_mx_dequantize(*q, 0, x)
    assert torch.equal(x.cpu(), ref.values(*q, 3, 300, 0).to(BF))
    del buf, x
    rows, cols = (1 << 21) + 77, 2048
    x = torch.ones(rows, cols, dtype=BF, device="cuda")
    x[-1] = torch.randn(cols, device="cuda")
    q = buffers(ss, rows, cols, 1)
    ss.ss_mx_quantize(x, 1, *q)
    last = ref.quantise(x[-1:], 1)[3]
    ss.ss_mx_dequantize(*q, 1, x)
    assert torch.equal(x[-1:].cpu().double(), last) and bool((x[:-1] == 1).all())


@gpu
@pytest.mark.parametrize("format,dtype,extra", [(0, BF, 0), (1, BF, 5), (0, F32, 3), (1, F32, 4)])
def test_a_large_matrix_is_its_parts(ss, format, dtype, extra):
    """A matrix large enough for whole tiles a CTA gives the bits of its pieces of 384 rows, which are not."""
    rows, cols = 10007, 2101
    gen = torch.Generator("cuda").manual_seed(3)
    x = randn(rows, cols, dtype, gen, extra=extra)
    q = buffers(ss, rows, cols, format)
    ss.ss_mx_quantize(x, format, *q)
    out, buf = matrix(rows, cols, dtype, extra, 0, fill=5.0)
    ss.ss_mx_dequantize(*q, format, out)
    assert outside_kept(buf, out, 5.0)
    data, scales = ss.ss_mx_bytes(rows, cols, format)
    pitch, tile = data // rows, scales // (-(-rows // 128))
    for r0 in range(0, rows, 384):
        n = min(384, rows - r0)
        p = buffers(ss, n, cols, format)
        ss.ss_mx_quantize(x[r0:r0 + n], format, *p)
        assert torch.equal(q[0][r0 * pitch:(r0 + n) * pitch], p[0][:n * pitch])
        t0, tiles = r0 // 128 * tile, -(-n // 128) * tile
        assert torch.equal(q[1][t0:t0 + tiles], p[1][:tiles])
        back = torch.empty(n, cols, dtype=dtype, device="cuda")
        ss.ss_mx_dequantize(*p, format, back)
        assert torch.equal(back, out[r0:r0 + n])


@gpu
def test_empty_matrices(ss):
    x, none = torch.empty(0, 64, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    n = ss.ss_launch_count()
    ss.ss_mx_quantize(x, 0, none, none)
    ss.ss_mx_dequantize(none, none, 0, x)
    q = buffers(ss, 5, 64, 0)
    ss.ss_mx_matmul(none, none, *q, 64, 0, torch.empty(0, 5, device="cuda"))
    ss.ss_mx_matmul(*q, none, none, 64, 0, torch.empty(5, 0, device="cuda"))
    assert ss.ss_launch_count() == n


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def quantised(ss, rows, cols, format, gen, wide=True):
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    if wide:
        x *= torch.exp2(2 * torch.randn(rows, cols, generator=gen, device="cuda"))
    q = buffers(ss, rows, cols, format)
    ss.ss_mx_quantize(x, format, *q)
    v = torch.empty(rows, cols, device="cuda")
    ss.ss_mx_dequantize(*q, format, v)
    return q, v.double()


def check_product(out, a, b):
    """Against the product of the values, with the bound at the file's head."""
    K = a.shape[1]
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = (K / 32 + 10) * 2.0 ** -22 * size + 1.01 * torch.finfo(out.dtype).eps / 2 * want.abs()
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), (float((off / tol.clamp(min=1e-300)).max()), torch.nonzero(~(off <= tol))[:8].tolist())


SIZES = [(1, 1, 1), (1, 128, 32), (1, 11008, 4096), (16, 256, 128), (17, 33, 65), (3, 777, 1001), (33, 130, 257),
         (64, 500, 384), (65, 129, 129), (130, 129, 640), (200, 40, 1024), (1000, 7, 300), (256, 256, 2048),
         (1021, 777, 1001), (5, 300, 20000), (2003, 72, 2688), (72, 1501, 520), (300, 64, 1100), (128, 2048, 2048),
         (40, 515, 5632), (1, 4099, 1100)]


@gpu
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(ss, format, M, N, K):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    (qa, a), (qb, b) = quantised(ss, M, K, format, gen), quantised(ss, N, K, format, gen)
    for dtype, extra, offset in ((BF, 0, 0), (F32, 0, 0), (BF, 3, 1)):
        out, buf = matrix(M, N, dtype, extra, offset, fill=5.0)
        ss.ss_mx_matmul(*qa, *qb, K, format, out)
        check_product(out, a, b)
        assert outside_kept(buf, out, 5.0)


@gpu
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K", [(2500, 2600, 300), (4097, 2049, 520), (1700, 7000, 64), (2048, 5632, 2048)])
def test_large_product(ss, format, M, N, K):
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    (qa, a), (qb, b) = quantised(ss, M, K, format, gen), quantised(ss, N, K, format, gen)
    for dtype, extra, offset in ((BF, 0, 0), (F32, 4, 0), (BF, 5, 3), (F32, 1, 1)):
        out, buf = matrix(M, N, dtype, extra, offset, fill=5.0)
        ss.ss_mx_matmul(*qa, *qb, K, format, out)
        check_product(out, a, b)
        assert outside_kept(buf, out, 5.0)


@gpu
@pytest.mark.parametrize("format", FORMATS)
@pytest.mark.parametrize("M,N,K", [(5, 300, 200), (200, 9, 200), (2500, 2600, 200)])
def test_product_keeps_special_values_in_their_row(ss, format, M, N, K):
    """A NaN block makes its row (or column) NaN and no other; scales far apart come through."""
    gen = torch.Generator("cuda").manual_seed(7)
    x, w = torch.randn(M, K, generator=gen, device="cuda"), torch.randn(N, K, generator=gen, device="cuda")
    x[3, 100], w[N - 1, 199] = math.nan, math.inf
    x[0] *= 2.0 ** -100
    w[0] *= 2.0 ** 100
    qa, qb = buffers(ss, M, K, format), buffers(ss, N, K, format)
    ss.ss_mx_quantize(x, format, *qa)
    ss.ss_mx_quantize(w, format, *qb)
    out = torch.empty(M, N, device="cuda")
    ss.ss_mx_matmul(*qa, *qb, K, format, out)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3], bad[:, N - 1] = True, True
    assert torch.equal(torch.isnan(out), bad)
    a, b = (ref.values(*q, r, K, format).cuda() for q, r in ((qa, M), (qb, N)))
    rows = [r for r in range(M) if r != 3]
    check_product(out[rows][:, :N - 1], a[rows], b[:N - 1])


@gpu
def test_the_same_bits_again_and_captured(ss):
    gen = torch.Generator("cuda").manual_seed(1)
    for M, N, K in ((3, 2048, 4096), (2500, 2600, 300)):
        (qa, a), (qb, b) = quantised(ss, M, K, 0, gen), quantised(ss, N, K, 0, gen)
        first, out = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        ss.ss_mx_matmul(*qa, *qb, K, 0, first)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ss.ss_mx_matmul(*qa, *qb, K, 0, out)
        side.synchronize()
        assert torch.equal(out, first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ss.ss_mx_matmul(*qa, *qb, K, 0, out)
        for _ in range(3):
            out.fill_(9.0)
            graph.replay()
            assert torch.equal(out, first)


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("rows,cols", [(1, 2048), (50, 64), (130, 1001), (300, 4096), (3, 16400)])
def test_norm_in_8_bits(ss, rows, cols):
    """The norm's own quantised output.  It rounds fp32 values that a 64-bit form can only bracket, so each element has
    to be what one of the values within the norm's error (60 w) gives, and the scale one of theirs."""
    gen = torch.Generator("cuda").manual_seed(rows)
    x, r = (torch.randn(rows, cols, generator=gen, device="cuda").to(BF) for _ in range(2))
    w = (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(BF)
    q, out, h = buffers(ss, rows, cols, 1), torch.empty_like(x), torch.empty_like(x)
    ss.ss_rms_norm(x, w, 1e-5, out=out, residual=r, sum_out=h, mx_data=q[0], mx_scales=q[1])
    hd = h.double()
    y = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + 1e-5) * w.double()
    lo, hi = (ref.quantise(y * (1 + s * 60 * 2.0 ** -24), 1) for s in (-1, 1))
    code, sign, byte = ref.unpack(*q, rows, cols, 1)
    blocks = lo[2].shape[1]
    assert bool(((byte[:, :blocks] == lo[2]) | (byte[:, :blocks] == hi[2])).all()) and bool((byte[:, blocks:] == 0).all())
    same = (lo[2] == hi[2]).repeat_interleave(32, 1)[:, :cols]
    ok = (code[:, :cols] == lo[0]) | (code[:, :cols] == hi[0])
    assert bool(ok[same].all()) and bool((code[:, cols:] == 0).all())
    live = code[:, :cols] != 0
    assert torch.equal(sign[:, :cols][live], (y.cpu() < 0)[live])
    plain = torch.empty_like(x)
    ss.ss_rms_norm(x, w, 1e-5, out=plain, residual=r)
    assert torch.equal(plain, out)


@gpu
def test_a_block_from_the_embedding_to_the_clipped_gradient(ss):
    """Dropout, residual, norm in 8 bits, a projection, the loss on the stream's norm, and all the way back: each call
    on what the one before left, against the formulas on the same quantised operands."""
    T, D, F, V = 300, 192, 520, 1000
    gen = torch.Generator("cuda").manual_seed(2)

    def rand(rows, cols, std):
        return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(BF)
    x, res = rand(T, D, 1.0), rand(T, D, 1.0)
    up, down, head = rand(F, D, 0.05), rand(D, F, 0.05), rand(V, D, 0.2)
    w1, w2 = (1 + rand(1, D, 0.2)[0] for _ in range(2))
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    rng = rng_of(11, 0)
    fmt = ss.SS_MXFP8
    h1, h2, y2 = (torch.empty_like(x) for _ in range(3))
    r1, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    q1, qup, tup = buffers(ss, T, D, fmt), buffers(ss, F, D, fmt), buffers(ss, D, F, fmt)
    a, qa, ta = torch.empty(T, F, dtype=BF, device="cuda"), buffers(ss, T, F, fmt), buffers(ss, F, T, fmt)
    qdown, tdown, z = buffers(ss, D, F, fmt), buffers(ss, F, D, fmt), torch.empty(T, D, dtype=BF, device="cuda")
    # forward
    ss.ss_rms_norm(x, w1, 1e-5, residual=res, sum_out=h1, rstd_out=r1, mx_data=q1[0], mx_scales=q1[1], dropout=0.1, rng=rng)
    ss.ss_mx_quantize(up, fmt, *qup, *tup)
    ss.ss_mx_matmul(*q1, *qup, D, fmt, a)
    ss.ss_mx_quantize(a, fmt, *qa, *ta)
    ss.ss_mx_quantize(down, fmt, *qdown, *tdown)
    ss.ss_mx_matmul(*qa, *qdown, F, fmt, z)
    rng2 = rng_of(11, 1)
    ss.ss_rms_norm(z, w2, 1e-5, out=y2, residual=h1, sum_out=h2, rstd_out=r2, dropout=0.1, rng=rng2)
    loss, dy2, dhead = torch.empty(1, device="cuda"), torch.empty_like(y2), torch.empty_like(head)
    ws = torch.empty(ss.ss_linear_ce_workspace(T, D, V, True), dtype=torch.uint8, device="cuda")
    ss.ss_linear_cross_entropy(y2, head, targets, loss, ws, d_hidden=dy2, d_weight=dhead)
    # backward
    nws = torch.empty(ss.ss_rms_norm_workspace(T, D), dtype=torch.uint8, device="cuda")
    dh2, dz, dw2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w2)
    ss.ss_rms_norm_backward(dy2, h2, w2, r2, dh2, nws, d_x=dz, d_weight=dw2, dropout=0.1, rng=rng2)
    rng3 = rng_of(11, 2)
    qz, tz = buffers(ss, T, D, fmt), buffers(ss, D, T, fmt)
    da, ddown = torch.empty_like(a), torch.empty_like(down)
    ss.ss_mx_quantize(dz, fmt, *qz, *tz, rng=rng3)
    ss.ss_mx_matmul(*qz, *tdown, D, fmt, da)
    ss.ss_mx_matmul(*tz, *ta, T, fmt, ddown)
    # against the formulas, on the operands as they were quantised
    val = lambda q, r, c: ref.values(*q, r, c, fmt).cuda()
    check_product(a, val(q1, T, D), val(qup, F, D))
    check_product(z, val(qa, T, F), val(qdown, D, F))
    check_product(da, val(qz, T, D), val(tdown, F, D))
    check_product(ddown, val(tz, D, T), val(ta, F, T))
    y = h2.double() / torch.sqrt(h2.double().square().mean(1, keepdim=True) + 1e-5) * w2.double()
    logp = torch.log_softmax(y2.double() @ head.double().t(), 1)
    assert abs(float(loss) + float(logp.gather(1, targets[:, None]).mean())) < 1e-4
    assert bool(((y2.double() - y).abs() <= 2.0 ** -8 * 1.05 * y.abs()).all())
    # what the whole path computes is near what it would be without quantisation: 8 bits a number, 2^-4 each at most
    keep1, keep2 = (ref.keep_mask(r, T, D, 0.1).cuda() for r in (rng, rng2))
    d = round(0.1 * 65536) / 65536
    f1 = torch.where(keep1, x.double() / (1 - d), 0.0) + res.double()
    n1 = f1 / torch.sqrt(f1.square().mean(1, keepdim=True) + 1e-5) * w1.double()
    f2 = torch.where(keep2, n1 @ up.double().t() @ down.double().t() / (1 - d), 0.0) + f1
    assert float((h2.double() - f2).norm() / f2.norm()) < 0.0625
    grads = [dhead, dw2, ddown]
    norm, cws = torch.empty(2, device="cuda"), torch.empty(ss.SS_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    ss.ss_clip_grads(grads, want / 2, norm, cws)
    assert abs(float(norm[0]) - want) <= 1e-5 * want and abs(float(norm[1]) - 0.5) <= 1e-5


@gpu
def test_refusals_of_the_binding(ss):
    x = torch.zeros(4, 64, device="cuda")
    q, t = buffers(ss, 4, 64, 0), buffers(ss, 64, 4, 0)
    out = torch.zeros(4, 4, device="cuda")
    bad = [lambda: ss.ss_mx_quantize(x, 0), lambda: ss.ss_mx_quantize(x, 3, *q), lambda: ss.ss_mx_quantize(x.half(), 0, *q),
           lambda: ss.ss_mx_quantize(x, 0, q[0]), lambda: ss.ss_mx_quantize(x.cpu(), 0, *q),
           lambda: ss.ss_mx_quantize(x, 0, q[0][:100], q[1]), lambda: ss.ss_mx_quantize(x, 0, q[0], q[1][:511]),
           lambda: ss.ss_mx_quantize(x, 0, q[0].float(), q[1]), lambda: ss.ss_mx_quantize(x, 0, q[0].cpu(), q[1]),
           lambda: ss.ss_mx_quantize(x, 0, *q, *[b[:256] for b in t]), lambda: ss.ss_mx_quantize(x[0], 0, *q),
           lambda: ss.ss_mx_quantize(x, 0, q[0][4:], q[1]), lambda: ss.ss_mx_quantize(x, 0, *q, rng=rng_of()[:1]),
           lambda: ss.ss_mx_dequantize(*q, 0, x.half()), lambda: ss.ss_mx_dequantize(q[0], None, 0, x),
           lambda: ss.ss_mx_dequantize(None, None, 0, x), lambda: ss.ss_mx_dequantize(*q, 0, x.t()),
           lambda: ss.ss_mx_matmul(*q, *q, 64, 0, out.half()), lambda: ss.ss_mx_matmul(*q, *q, 0, 0, out),
           lambda: ss.ss_mx_matmul(*q, *q, 300, 0, out), lambda: ss.ss_mx_matmul(*q, None, None, 64, 0, out),
           lambda: ss.ss_mx_matmul(*q, *q, 64, 1, torch.zeros(40, 4, device="cuda")),
           lambda: ss.ss_mx_matmul(*q, *q, 64, 0, out.cpu()), lambda: ss.ss_mx_matmul(*q, *q, 64, 0, out[:, ::2])]
    for k, call in enumerate(bad):
        with pytest.raises(ss.ShardStateError):
            call()
            pytest.fail(f"call {k} was not refused")
