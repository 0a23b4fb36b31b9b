"""Dropout and the residual stream's norm against the formulas in 64 bits.

Tolerances.  u is half a step of the type (bf16 2^-8, fp32 2^-24, relative), w = 2^-24.  Sums over a row are taken
by at most 512 threads, 64 elements each in turn, then 5 adds in the warp and 16 over the warps, or by up to 1024 of at
most 16 elements and 32 warps: a term passes at most 64 + 5 + 16 adds, and its product's rounding, so the sum is off by at
most SUM = 90 w times the sum of the terms' magnitudes (their sum itself for squares).
"""
import math

import pytest
import torch

from tests.stream_reference import keep_mask, philox

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
W = 2.0 ** -24
SUM = 90 * W


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(scope="module")
def ss():
    import __graft_entry__
    __graft_entry__.build()
    import sharded_state_gb300 as ss
    return ss


def matrix(rows, cols, dtype, extra=0, offset=0, fill=3.0):
    """A [rows, cols] view with row stride cols + extra, `offset` elements past a 16-byte boundary, and its buffer."""
    buf = torch.full((16 + offset + rows * (cols + extra) + 16,), fill, dtype=dtype, device="cuda")
    return buf[16 + offset:16 + offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols], buf


def randn(rows, cols, dtype, gen, std=1.0, **kw):
    m, _ = matrix(rows, cols, dtype, **kw)
    m.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * std)
    return m


def outside_kept(buf, view, fill):
    """Whether the buffer around a view is as it was."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[mask] == fill).all())


def block(layout, fields, changed):
    """An argument block of the C ABI, some of its fields changed."""
    assert set(changed) <= set(fields)
    return layout.pack(*(0 if v is None else v for v in {**fields, **changed}.values()))


def rng_of(seed=12345, offset=77):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def dropped(x, mask, p):
    d = round(p * 65536) / 65536
    return torch.where(mask.to(x.device), x.double() / (1 - d), 0.0)


# ---------------------------------------------------------------------------
# on the CPU
# ---------------------------------------------------------------------------

def test_generator_known_answers():
    """The published vectors of Philox4x32-10, on the form the other tests compare with."""
    assert philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert philox([ones] * 4, [ones] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_refusals_of_the_c_calls(ss):
    """Argument errors come back as status codes, before anything is launched."""
    import ctypes
    lib, n = ss.lib(), ss.ss_launch_count()
    a = 4096  # an aligned address that nothing reads

    def drop(rows=4, cols=8, eb=2, x=a, ldx=8, out=a, ldo=8, p=0.5, rng=a):
        return lib.ss_dropout(rows, cols, eb, x, ldx, out, ldo, p, rng, None)
    assert drop(rows=-1) == drop(cols=-1) == drop(eb=3) == drop(x=None) == drop(out=None) == ss.SS_EINVAL
    assert drop(p=1.0) == drop(p=-0.1) == drop(p=math.nan) == drop(p=1 - 2.0 ** -18) == drop(rng=None) == ss.SS_EINVAL
    assert drop(ldx=7) == drop(ldo=7) == ss.SS_EINVAL
    assert drop(x=a + 1) == drop(out=a + 1) == drop(rng=a + 4) == drop(eb=4, x=a + 2) == ss.SS_EALIGN
    assert drop(rows=1 << 31) == drop(ldx=1 << 60) == drop(rows=1, cols=1 << 36, ldx=1 << 36, ldo=1 << 36) == ss.SS_EOVERFLOW
    assert drop(rows=0, x=None, out=None) == drop(cols=0, ldx=0, ldo=0) == ss.SS_OK

    def norm(**kw):
        s = dict(rows=4, cols=8, elem_bytes=2, x=a, x_stride=8, residual=a, residual_stride=8, weight=a, eps=1e-5,
                 dropout=0.0, rng=None, sum_out=a, sum_stride=8, out=a, out_stride=8, rstd_out=a, mx_data=a, mx_scales=a)
        return lib.ss_rms_norm(block(ss._NORM, s, kw), None)
    none = dict(sum_out=None, out=None, rstd_out=None, mx_data=None, mx_scales=None)
    assert norm(rows=-1) == norm(cols=0) == norm(elem_bytes=8) == norm(x=None) == norm(weight=None) == ss.SS_EINVAL
    assert norm(eps=-1.0) == norm(eps=math.inf) == norm(eps=math.nan) == norm(eps=1e300) == norm(**none) == ss.SS_EINVAL
    assert norm(mx_data=None) == norm(mx_scales=None) == norm(dropout=0.5) == norm(dropout=1.0, rng=a) == ss.SS_EINVAL
    assert norm(x_stride=7) == norm(residual_stride=7) == norm(sum_stride=7) == norm(out_stride=7) == ss.SS_EINVAL
    assert norm(cols=32769, x_stride=32769, residual_stride=32769) == norm(rows=1 << 31) == norm(x_stride=1 << 62) == ss.SS_EOVERFLOW
    for field in ("x", "residual", "weight", "sum_out", "out", "rstd_out", "mx_data", "mx_scales"):
        assert norm(**{field: a + 1}) == ss.SS_EALIGN, field
    assert norm(rows=0, **none) == ss.SS_OK and lib.ss_rms_norm(None, None) == ss.SS_EINVAL

    def grad(**kw):
        s = dict(rows=4, cols=8, elem_bytes=2, d_out=a, d_out_stride=8, h=a, h_stride=8, weight=a, rstd=a, d_sum=a,
                 d_sum_stride=8, dropout=0.0, rng=None, d_h=a, d_h_stride=8, d_x=a, d_x_stride=8, d_weight=a, workspace=a,
                 workspace_bytes=1 << 20)
        return lib.ss_rms_norm_backward(block(ss._NORM_GRAD, s, kw), None)
    assert grad(rows=-1) == grad(cols=0) == grad(elem_bytes=1) == grad(d_out=None) == grad(h=None) == ss.SS_EINVAL
    assert grad(weight=None) == grad(rstd=None) == grad(workspace=None) == grad(workspace_bytes=31) == ss.SS_EINVAL
    assert grad(d_h=None, d_x=None, d_weight=None) == grad(dropout=0.5) == grad(d_sum_stride=7) == ss.SS_EINVAL
    assert grad(d_out_stride=7) == grad(h_stride=7) == grad(d_h_stride=7) == grad(d_x_stride=7) == ss.SS_EINVAL
    for field in ("d_out", "h", "weight", "rstd", "d_sum", "d_h", "d_x", "d_weight", "workspace"):
        assert grad(**{field: a + 1}) == ss.SS_EALIGN, field
    assert grad(cols=32769, d_out_stride=40000, h_stride=40000) == grad(rows=1 << 31) == ss.SS_EOVERFLOW
    assert grad(rows=0, d_weight=None) == ss.SS_OK and lib.ss_rms_norm_backward(None, None) == ss.SS_EINVAL
    size = ctypes.c_size_t()
    assert lib.ss_rms_norm_workspace(4, 0, ctypes.byref(size)) == lib.ss_rms_norm_workspace(4, 8, None) == ss.SS_EINVAL
    assert lib.ss_rms_norm_workspace(4, 1 << 20, ctypes.byref(size)) == ss.SS_EOVERFLOW
    assert ss.ss_launch_count() == n


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,extra,offset,p", [
    (1, 1, 0, 0, 0.5), (3, 7, 0, 0, 0.1), (50, 64, 0, 0, 0.1), (33, 513, 0, 3, 0.25), (17, 1001, 24, 1, 0.9),
    (129, 24, 8, 0, 0.0), (5, 11008, 0, 0, 1 - 2.0 ** -16), (1, 70001, 0, 0, 0.3), (2000, 9, 0, 0, 0.5)])
def test_dropout(ss, dtype, rows, cols, extra, offset, p):
    gen = torch.Generator("cuda").manual_seed(rows * cols)
    x = randn(rows, cols, dtype, gen, extra=extra, offset=offset)
    out, buf = matrix(rows, cols, dtype, extra, offset, fill=5.0)
    rng = rng_of(-3, (1 << 62) + 5)
    ss.ss_dropout(x, out, p, rng)
    want = dropped(x, keep_mask(rng, rows, cols, p), p)
    # the factor in fp32, the product, the result
    assert bool(((out.double() - want).abs() <= (half_step(dtype) + 3 * W) * want.abs()).all())
    assert bool(((out == 0) == (want == 0)).all())
    assert outside_kept(buf, out, 5.0)
    twice = x.clone()
    ss.ss_dropout(twice, twice, p, rng)
    assert torch.equal(twice, out)


@gpu
def test_dropout_drops_whatever_was_there(ss):
    x = torch.full((4, 640), math.nan, device="cuda")
    x[1] = math.inf
    out, rng = torch.empty_like(x), rng_of()
    ss.ss_dropout(x, out, 0.5, rng)
    keep = keep_mask(rng, 4, 640, 0.5).cuda()
    assert bool((out[~keep] == 0).all()) and bool(torch.isnan(out[keep & torch.isnan(x)]).all())
    assert bool(torch.isinf(out[1][keep[1]]).all())


@gpu
def test_dropout_at_offsets_past_32_bits(ss):
    """Two rows more than 2^32 bytes apart, and one row of more than 2^31 elements."""
    stride = (1 << 31) + 24
    buf = torch.ones(stride + 4096, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (2, 4096), (stride, 1))
    rng = rng_of()
    ss.ss_dropout(x, x, 0.5, rng)
    assert torch.equal(x != 0, keep_mask(rng, 2, 4096, 0.5).cuda())
    assert bool((buf[4096:8192] == 1).all())
    n = (1 << 31) + 1003
    x = torch.ones(1, n, dtype=BF, device="cuda")
    ss.ss_dropout(x, x, 0.25, rng)
    at = (1 << 31) - 8
    assert torch.equal(x[:, at:] != 0, keep_mask(rng, 1, n - at, 0.25, col0=at).cuda())


# ---------------------------------------------------------------------------
# the norm
# ---------------------------------------------------------------------------

class Norm:
    """One forward call and what it should have given."""

    def __init__(self, ss, rows, cols, dtype, p=0.0, residual=True, extra=0, offset=0, eps=1e-5, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        kw = dict(extra=extra, offset=offset)
        self.rows, self.cols, self.dtype, self.p, self.eps = rows, cols, dtype, p, eps
        self.x = randn(rows, cols, dtype, gen, **kw)
        self.residual = randn(rows, cols, dtype, gen, 2.0, **kw) if residual else None
        self.weight = (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
        self.rng = rng_of(seed, 9) if p else None
        self.h, self.hbuf = matrix(rows, cols, dtype, fill=5.0, **kw)
        self.out, self.obuf = matrix(rows, cols, dtype, fill=5.0, **kw)
        self.rstd = torch.full((rows,), 9.0, device="cuda")
        self.kw = kw
        ss.ss_rms_norm(self.x, self.weight, eps, out=self.out, residual=self.residual, sum_out=self.h,
                       rstd_out=self.rstd, dropout=p, rng=self.rng)

    def check(self):
        x = self.x.double()
        if self.p:
            x = dropped(self.x, keep_mask(self.rng, self.rows, self.cols, self.p), self.p)
        r = self.residual.double() if self.residual is not None else torch.zeros_like(x)
        h = self.h.double()
        tol = half_step(self.dtype) * (x + r).abs() * 1.01 + 4 * W * (x.abs() + r.abs())
        assert bool(((h - (x + r)).abs() <= tol).all())
        rstd = 1 / torch.sqrt(h.square().mean(1) + self.eps)  # the sum's error halves under the root
        got = self.rstd.double()
        assert bool(((got - rstd).abs() <= (SUM / 2 + 4 * W) * rstd).all()), float(((got - rstd) / rstd).abs().max() / W)
        out = h * rstd[:, None] * self.weight.double()
        tol = (half_step(self.dtype) * 1.01 + SUM / 2 + 6 * W) * out.abs()
        assert bool(((self.out.double() - out).abs() <= tol).all())
        assert outside_kept(self.hbuf, self.h, 5.0) and outside_kept(self.obuf, self.out, 5.0)
        return self

    def backward(self, ss, d_sum=True, seed=1, scale=1e-2):
        gen = torch.Generator("cuda").manual_seed(seed)
        rows, cols, dtype = self.rows, self.cols, self.dtype
        self.dy = randn(rows, cols, dtype, gen, scale, **self.kw)
        self.ds = randn(rows, cols, dtype, gen, scale, **self.kw) if d_sum else None
        self.dh, self.dhbuf = matrix(rows, cols, dtype, fill=5.0, **self.kw)
        self.dx, self.dxbuf = matrix(rows, cols, dtype, fill=5.0, **self.kw)
        self.dw = torch.full((cols + 2,), 5.0, dtype=dtype, device="cuda")
        ws = torch.full((ss.ss_rms_norm_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
        ss.ss_rms_norm_backward(self.dy, self.h, self.weight, self.rstd, self.dh, ws, d_sum=self.ds, d_x=self.dx,
                                d_weight=self.dw[:cols], dropout=self.p, rng=self.rng)
        return self

    def check_backward(self):
        dy, h, w, r = (t.double() for t in (self.dy, self.h, self.weight, self.rstd))
        n = h * r[:, None]
        g = dy * w
        ds = self.ds.double() if self.ds is not None else torch.zeros_like(g)
        mean, size = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
        want = r[:, None] * (g - n * mean) + ds
        # the mean carries SUM and its terms' 3 roundings; then 6 more of either term
        tol = r[:, None] * (n.abs() * size * (SUM + 4 * W) + 6 * W * (g.abs() + n.abs() * mean.abs())) + 4 * W * ds.abs()
        top = half_step(self.dtype) * 1.01
        assert bool(((self.dh.double() - want).abs() <= tol + top * want.abs()).all())
        dx, slack = want, tol
        if self.p:
            mask = keep_mask(self.rng, self.rows, self.cols, self.p)
            dx, slack = dropped(want, mask, self.p), dropped(tol, mask, self.p)
        assert bool(((self.dx.double() - dx).abs() <= slack + (top + 3 * W) * dx.abs()).all())
        dw, terms = (dy * n).sum(0), (dy * n).abs().sum(0)
        # rows in turn, then over the teams, then over the CTAs: never more adds than there are rows
        tol = (self.rows + 4) * W * terms + top * dw.abs()
        assert bool(((self.dw[:self.cols].double() - dw).abs() <= tol).all())
        assert bool((self.dw[self.cols:] == 5).all())
        assert outside_kept(self.dhbuf, self.dh, 5.0) and outside_kept(self.dxbuf, self.dx, 5.0)
        return self


SIZES = [(1, 1), (1, 2048), (3, 7), (50, 64), (700, 17), (33, 513), (5, 1001), (301, 2048), (2, 4095), (9, 4096),
         (700, 1030), (7, 5632), (5, 11008), (3, 16384), (2, 16391), (2, 32768),
         (40, 5632), (20, 8192), (9, 9589), (11, 20000),
         (20, 5155), (9, 6001)]


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_and_gradient(ss, rows, cols, dtype):
    Norm(ss, rows, cols, dtype, p=0.1).check().backward(ss).check_backward()


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("extra,offset", [(8, 0), (0, 1), (3, 0), (13, 5), (1, 2)])
def test_norm_strides(ss, dtype, extra, offset):
    Norm(ss, 37, 1000, dtype, p=0.3, extra=extra, offset=offset).check().backward(ss).check_backward()


@gpu
@pytest.mark.parametrize("p,residual", [(0.0, True), (0.0, False), (0.5, False)])
def test_norm_without(ss, p, residual):
    n = Norm(ss, 65, 520, BF, p=p, residual=residual).check().backward(ss, d_sum=residual).check_backward()
    if not p:
        assert torch.equal(n.dx, n.dh)


@gpu
def test_norm_of_no_rows(ss):
    n = Norm(ss, 0, 96, BF, p=0.1).backward(ss)
    assert bool((n.dw[:96] == 0).all())


@gpu
def test_outputs_are_optional_and_in_place(ss):
    """Every subset of the outputs gives the same bits, and so does the stream updated in place."""
    n = Norm(ss, 67, 1000, BF, p=0.2)
    kw = dict(dropout=0.2, rng=n.rng)
    out = torch.empty_like(n.out)
    ss.ss_rms_norm(n.x, n.weight, n.eps, out=out, residual=n.residual, **kw)
    assert torch.equal(out, n.out)
    h = torch.empty_like(n.h)
    ss.ss_rms_norm(n.x, n.weight, n.eps, residual=n.residual, sum_out=h, **kw)
    assert torch.equal(h, n.h)
    rstd = torch.empty_like(n.rstd)
    ss.ss_rms_norm(n.x, n.weight, n.eps, residual=n.residual, rstd_out=rstd, **kw)
    assert torch.equal(rstd, n.rstd)
    x, r = n.x.clone(), n.residual.clone()
    ss.ss_rms_norm(x, n.weight, n.eps, out=x, residual=r, sum_out=r, **kw)
    assert torch.equal(x, n.out) and torch.equal(r, n.h)
    x = n.x.clone()
    ss.ss_rms_norm(x, n.weight, n.eps, residual=n.residual, sum_out=x, **kw)
    assert torch.equal(x, n.h)
    n.backward(ss)
    for name in ("ds", "dy"):
        t = getattr(n, name).clone()
        ss.ss_rms_norm_backward(t if name == "dy" else n.dy, n.h, n.weight, n.rstd, t, None,
                                d_sum=t if name == "ds" else n.ds, **kw)
        assert torch.equal(t, n.dh), name
    dx = torch.empty_like(n.dx)
    ss.ss_rms_norm_backward(n.dy, n.h, n.weight, n.rstd, None, None, d_sum=n.ds, d_x=dx, **kw)
    assert torch.equal(dx, n.dx)
    dw, ws = torch.empty_like(n.weight), torch.empty(ss.ss_rms_norm_workspace(67, 1000), dtype=torch.uint8, device="cuda")
    ss.ss_rms_norm_backward(n.dy, n.h, n.weight, n.rstd, None, ws, d_weight=dw, **kw)
    assert torch.equal(dw, n.dw[:1000])


@gpu
def test_norm_and_dropout_share_a_mask(ss):
    """The norm's dropout is ss_dropout's: the sum of its output and the residual is h, bit for bit."""
    n = Norm(ss, 41, 777, F32, p=0.4)
    x = torch.empty(41, 777, device="cuda")
    ss.ss_dropout(n.x, x, 0.4, n.rng)
    assert torch.equal(x + n.residual, n.h)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_with_special_values(ss, dtype):
    """NaN and infinities stay in their rows; a row of zeros is zeros."""
    x = torch.randn(5, 300, device="cuda").to(dtype)
    plain = x.clone()
    x[1, 7], x[2, 299], x[3] = math.nan, -math.inf, 0
    w, eps = torch.ones(300, dtype=dtype, device="cuda"), 1e-6
    out, ref = torch.empty_like(x), torch.empty_like(x)
    ss.ss_rms_norm(x, w, eps, out=out)
    ss.ss_rms_norm(plain, w, eps, out=ref)
    assert torch.equal(out[[0, 4]], ref[[0, 4]]) and bool(torch.isnan(out[1]).all()) and bool((out[3] == 0).all())
    assert bool(torch.isnan(out[2, 299])) and bool((out[2, :299] == 0).all())


@gpu
def test_gradient_against_differences(ss):
    """<dx, v> against the loss at x +- e v, in fp32.  L = <out, dy> + <h, ds> along a line is smooth: with rows of
    about unit scale and elements of the direction of 4/3 at most (the dropout's factor), the third derivative of out is
    below 15 |h| (4/3)^3 rstd^3 < 500 an element; e = 2^-7 makes of it e^2 / 6 * 500 < 0.006 sum|dy|.  Each L is a sum in
    64 bits of fp32 outputs whose error is 100 w at most: 100 w sum|out dy| / e < 0.001 sum|out dy|."""
    n = Norm(ss, 24, 200, F32, p=0.25, seed=5).backward(ss, scale=1.0)
    gen = torch.Generator("cuda").manual_seed(3)
    v = (torch.rand(24, 200, generator=gen, device="cuda") > 0.5).float() * 2 - 1
    vw = (torch.rand(200, generator=gen, device="cuda") > 0.5).float() * 2 - 1
    e = 2.0 ** -7

    def loss(x, r, w):
        out, h = torch.empty_like(n.out), torch.empty_like(n.h)
        ss.ss_rms_norm(x, w, n.eps, out=out, residual=r, sum_out=h, dropout=n.p, rng=n.rng)
        return float((out.double() * n.dy.double()).sum() + (h.double() * n.ds.double()).sum())
    for got, lo, hi in (((n.dx.double() * v).sum(), (n.x - e * v, n.residual, n.weight), (n.x + e * v, n.residual, n.weight)),
                        ((n.dh.double() * v).sum(), (n.x, n.residual - e * v, n.weight), (n.x, n.residual + e * v, n.weight)),
                        ((n.dw[:200].double() * vw).sum(), (n.x, n.residual, n.weight - e * vw), (n.x, n.residual, n.weight + e * vw))):
        quotient = (loss(*hi) - loss(*lo)) / (2 * e)
        terms = 0.006 * float(n.dy.abs().sum()) + 0.001 * float((n.out * n.dy).abs().sum() + (n.h * n.ds).abs().sum())
        assert abs(float(got) - quotient) <= terms, (float(got), quotient, terms)


@gpu
def test_captured_and_on_another_stream(ss):
    """A captured forward and backward draw another mask once the offset on the device is another."""
    n = Norm(ss, 64, 320, BF, p=0.5)
    ws = torch.empty(ss.ss_rms_norm_workspace(64, 320), dtype=torch.uint8, device="cuda")
    dy, rng = torch.randn_like(n.x), rng_of(4, 1)
    out, h, rstd, dh, dx = (torch.empty_like(t) for t in (n.out, n.h, n.rstd, n.x, n.x))
    dw = torch.empty_like(n.weight)

    def step():
        ss.ss_rms_norm(n.x, n.weight, n.eps, out=out, residual=n.residual, sum_out=h, rstd_out=rstd, dropout=0.5, rng=rng)
        ss.ss_rms_norm_backward(dy, h, n.weight, rstd, dh, ws, d_x=dx, d_weight=dw, dropout=0.5, rng=rng)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for offset in (1, 2, 3):
        rng[1] = offset
        graph.replay()
        got = [t.clone() for t in (out, h, rstd, dh, dx, dw)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, h, rstd, dh, dx, dw)))
        assert torch.equal(dx != 0, keep_mask(rng, 64, 320, 0.5).cuda() & (dh != 0))


@gpu
def test_the_same_bits_again(ss):
    a, b = (Norm(ss, 2100, 1030, BF, p=0.1).backward(ss) for _ in range(2))
    for name in ("h", "out", "rstd", "dh", "dx", "dw"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@gpu
def test_two_calls_at_once(ss):
    """Calls on two streams, each with its own workspace, give what they give alone."""
    a, b = Norm(ss, 900, 2048, BF, p=0.1, seed=1), Norm(ss, 1100, 1000, BF, p=0.2, seed=2)
    want = [(n.backward(ss).dh.clone(), n.dw.clone()) for n in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for n in (a, b):
        ws = torch.empty(ss.ss_rms_norm_workspace(n.rows, n.cols), dtype=torch.uint8, device="cuda")
        jobs.append((n, ws, torch.empty_like(n.dh), torch.empty_like(n.weight)))
    torch.cuda.synchronize()
    for _ in range(8):
        for stream, (n, ws, dh, dw) in zip(streams, jobs):
            ss.ss_rms_norm_backward(n.dy, n.h, n.weight, n.rstd, dh, ws, d_sum=n.ds, d_weight=dw, dropout=n.p, rng=n.rng,
                                    stream=stream)
    torch.cuda.synchronize()
    for (n, ws, dh, dw), (want_dh, want_dw) in zip(jobs, want):
        assert torch.equal(dh, want_dh) and torch.equal(dw, want_dw[:n.cols])


@gpu
def test_refusals_of_the_binding(ss):
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    rng, out = rng_of(), torch.zeros(4, 64, device="cuda")
    r = torch.zeros(4, device="cuda")
    bad = [lambda: ss.ss_dropout(x.cpu(), out, 0.5, rng), lambda: ss.ss_dropout(x, out.bfloat16(), 0.5, rng),
           lambda: ss.ss_dropout(x, out[:, :32], 0.5, rng), lambda: ss.ss_dropout(x.half(), out.half(), 0.5, rng),
           lambda: ss.ss_dropout(x, out, 0.5, rng.float()), lambda: ss.ss_dropout(x, out, 0.5, None),
           lambda: ss.ss_dropout(x, out, 0.5, rng.cpu()), lambda: ss.ss_dropout(x.t(), out.t(), 0.5, rng),
           lambda: ss.ss_dropout(x, out[:1].expand(4, 64), 0.5, rng), lambda: ss.ss_dropout(x[0], out[0], 0.5, rng),
           lambda: ss.ss_rms_norm(x, w, 1e-5), lambda: ss.ss_rms_norm(x, w[:63], 1e-5, out=out),
           lambda: ss.ss_rms_norm(x, w.bfloat16(), 1e-5, out=out), lambda: ss.ss_rms_norm(x, None, 1e-5, out=out),
           lambda: ss.ss_rms_norm(x, w, 1e-5, out=out, rstd_out=r[:3]),
           lambda: ss.ss_rms_norm(x, w, 1e-5, out=out, dropout=0.5),
           lambda: ss.ss_rms_norm(x, w, 1e-5, out=out, mx_data=torch.zeros(512, dtype=torch.uint8, device="cuda")),
           lambda: ss.ss_rms_norm_backward(x, x, w, r, out, None, d_weight=w.clone()),
           lambda: ss.ss_rms_norm_backward(x, x, w, r, None, None),
           lambda: ss.ss_rms_norm_backward(x, x, w, r[:2], out, None),
           lambda: ss.ss_rms_norm_backward(x[:3], x, w, r, out, None)]
    for k, call in enumerate(bad):
        with pytest.raises(ss.ShardStateError):
            call()
            pytest.fail(f"call {k} was not refused")
