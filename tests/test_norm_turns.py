"""Dropout and the norm where a CTA takes rows in turn, and in every form that the kernels have.

What is compared, and how far it may be off, is tests/test_norm.py's: at most 1024 threads take a row, of 8 elements each
where they are more than 768, of 16 where they are more than 512 and of up to 64 else, so that a term passes 64 + 5 + 16 adds
at the most (8 + 5 + 32 at 1024 threads) and SUM holds; a weight gradient's term passes no more adds than there are rows.
Rows of a turn on 152 SMs: 2432 of up to 256 columns, 304 to 1216 of up to 4096, 152 of more.
"""
import pytest
import torch

from tests.stream_reference import keep_mask
from tests.test_norm import BF, F32, W, Norm, dropped, half_step, matrix, outside_kept, randn, rng_of, ss  # noqa: F401

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [
    # rows on 16 bytes: one load a thread, two, two of more than 256 threads, four, eight
    (5003, 128), (2500, 520), (1000, 2048), (700, 4096), (500, 5632), (400, 8192), (400, 12000), (400, 20000),
    # at odd addresses, as many loads of as many threads as each type has
    (5003, 131), (1300, 1999), (400, 2999), (400, 5155), (400, 7001), (400, 9589), (400, 11003), (400, 13001),
    (400, 16391)])
def test_rows_in_turn(ss, rows, cols, dtype):  # noqa: F811
    Norm(ss, rows, cols, dtype, p=0.1).check().backward(ss).check_backward()


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(330, 1001), (400, 4096), (200, 7001), (200, 8200), (200, 11003), (200, 13001),
                                       (200, 20000), (200, 20001)])
def test_rows_in_turn_in_place(ss, rows, cols, dtype):  # noqa: F811
    """Gradients over d_out or d_sum, and the stream over its input, give the bits that they give elsewhere, rows that
    are read twice among them."""
    n = Norm(ss, rows, cols, dtype, p=0.1).backward(ss)
    kw = dict(dropout=n.p, rng=n.rng)
    for name in ("ds", "dy"):
        t = getattr(n, name).clone()
        ss.ss_rms_norm_backward(t if name == "dy" else n.dy, n.h, n.weight, n.rstd, t, None,
                                d_sum=t if name == "ds" else n.ds, **kw)
        assert torch.equal(t, n.dh), name
    x, r = n.x.clone(), n.residual.clone()
    ss.ss_rms_norm(x, n.weight, n.eps, out=x, residual=r, sum_out=r, **kw)
    assert torch.equal(x, n.out) and torch.equal(r, n.h)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,extra,offset,out_extra,out_offset", [
    # more groups of 8 than a grid of 152 SMs has threads (311,296)
    (200003, 24, 0, 0, 0, 0), (200003, 24, 8, 0, 24, 0), (60000, 71, 0, 1, 0, 3), (60000, 71, 2, 0, 5, 7),
    # more pieces of 512 columns than it has warps (9728)
    (3001, 4096, 0, 0, 8, 0), (1500, 11008, 0, 0, 0, 0), (1500, 11003, 0, 3, 0, 0), (1500, 11003, 5, 0, 2, 1)])
def test_dropout_in_turn(ss, rows, cols, extra, offset, out_extra, out_offset, dtype):  # noqa: F811
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    x = randn(rows, cols, dtype, gen, extra=extra, offset=offset)
    out, buf = matrix(rows, cols, dtype, out_extra, out_offset, fill=5.0)
    rng = rng_of(17, 5)
    ss.ss_dropout(x, out, 0.25, rng)
    want = dropped(x, keep_mask(rng, rows, cols, 0.25), 0.25)
    assert bool(((out.double() - want).abs() <= (half_step(dtype) + 3 * W) * want.abs()).all())
    assert bool(((out == 0) == (want == 0)).all())
    assert outside_kept(buf, out, 5.0)


@gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols,here,there", [(1024, (0, 0), (24, 8)), (5632, (8, 0), (32, 16)), (1024, (1, 0), (3, 5)),
                                             (5155, (0, 0), (2, 1)), (9589, (0, 3), (7, 0))])
def test_the_same_bits_elsewhere(ss, cols, here, there, dtype):  # noqa: F811
    """Other addresses and strides give the same bits, as long as they are multiples of 16 bytes, or are not, alike."""
    a, b = (Norm(ss, 310, cols, dtype, p=0.1, extra=e, offset=o).backward(ss) for e, o in (here, there))
    for name in ("x", "dy", "h", "out", "rstd", "dh", "dx", "dw"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
