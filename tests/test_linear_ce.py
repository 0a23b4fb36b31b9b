"""Linear cross entropy and its gradients against the formulas in 64 bits.

Tolerances, for the bf16 inputs as they are.  A logit is a sum of D exact
products in the tensor cores' fp32 accumulator, 16 at a time: its error is at most
dl = (D / 16 + 2) * 2^-22 * sum_k |h_k w_k| (2^-22: an add that keeps 24 bits and
may truncate, twice over for the products' own alignment).  The loss is a
log-sum-exp minus one logit: 2 dl and a few fp32 roundings of either.  A gradient is
a sum of (p - [v = y]) x: p carries 2 dl and its rounding to bf16 (half an ulp of
8 significant bits: 2^-8), the sum its own fp32 error, the result another 2^-8.
"""
import math

import pytest
import torch

gpu = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ss():
    import __graft_entry__
    __graft_entry__.build()
    import sharded_state_gb300 as ss
    return ss


def strided(rows, cols, extra, offset, fill=3.0):
    """A [rows, cols] bf16 view with row stride cols + extra, `offset` elements past a
    16-byte boundary, and the buffer around it."""
    buf = torch.full((16 + offset + rows * (cols + extra) + 16,), fill, dtype=BF, device="cuda")
    return buf[16 + offset:16 + offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols], buf


class Case:
    def __init__(self, T, V, D, mask="none", h_extra=0, w_extra=0, offset=0, seed=0, std=0.5, ignore=-100):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.T, self.V, self.D, self.ignore = T, V, D, ignore
        self.h, self.hbuf = strided(T, D, h_extra, offset)
        self.w, self.wbuf = strided(V, D, w_extra, offset)
        self.h.copy_(torch.randn(T, D, generator=gen, device="cuda"))
        self.w.copy_(torch.randn(V, D, generator=gen, device="cuda") * std / math.sqrt(D) * 4)
        self.y = torch.randint(0, V, (T,), generator=gen, device="cuda")
        drop = {"none": [], "all": range(T), "all_but_last": range(T - 1), "alternate": range(0, T, 2),
                "first_half": range(T // 2),
                "random": torch.randperm(T, generator=gen, device="cuda")[:T // 3].tolist()}[mask]
        self.y[list(drop)] = ignore
        if ignore >= 0:  # no target is the ignored class by accident
            keep = torch.ones(T, dtype=torch.bool, device="cuda")
            keep[list(drop)] = False
            self.y[keep & (self.y == ignore)] = (ignore + 1) % V

    def run(self, ss, dh=True, dw=True, out_extra=0, out_offset=0, workspace=None, **kw):
        T, V, D = self.T, self.V, self.D
        self.loss = torch.full((1,), 99.0, device="cuda")
        self.token_loss = torch.full((T,), 99.0, device="cuda")
        self.dh, self.dhbuf = strided(T, D, out_extra, out_offset, fill=5.0) if dh else (None, None)
        self.dw, self.dwbuf = strided(V, D, out_extra, out_offset, fill=5.0) if dw else (None, None)
        aligned = self.w.data_ptr() % 16 == 0 and self.w.stride(0) % 8 == 0
        n = ss.ss_linear_ce_workspace(T, D, V, dh or dw, stage_weight=not aligned)
        ws = workspace if workspace is not None else torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
        ss.ss_linear_cross_entropy(self.h, self.w, self.y, self.loss, ws, token_loss_out=self.token_loss,
                                   d_hidden=self.dh, d_weight=self.dw, ignore_index=self.ignore, **kw)
        return self

    def check(self, reduction="mean", grad_scale=1.0):
        keep = torch.nonzero(self.y != self.ignore).squeeze(1)
        n = keep.numel()
        h, w, y = self.h[keep].double(), self.w.double(), self.y[keep]
        logits = h @ w.t()
        lse = torch.logsumexp(logits, 1)
        hit = logits.gather(1, y[:, None]).squeeze(1)
        size = h.abs() @ w.abs().t()
        dl = (self.D / 16 + 2) * 2.0 ** -22 * (size.amax(1) if n else size.sum(1))
        want = lse - hit
        tol = 2 * dl + 2.0 ** -22 * (lse.abs() + hit.abs() + 1)
        got = self.token_loss.double()
        assert bool(((got[keep] - want).abs() <= tol).all()), float(((got[keep] - want).abs() / tol).max())
        away = torch.ones(self.T, dtype=torch.bool, device="cuda")
        away[keep] = False
        assert bool((got[away] == 0).all())
        total = float(want.sum()) / (max(n, 1) if reduction == "mean" else 1)
        bound = float(tol.sum()) / (max(n, 1) if reduction == "mean" else 1) + 2.0 ** -23 * abs(total)
        assert abs(float(self.loss) - total) <= bound
        scale = grad_scale / (max(n, 1) if reduction == "mean" else 1)
        p = (logits - lse[:, None]).exp()
        hot = torch.zeros_like(p).scatter_(1, y[:, None], 1.0)
        d = (p - hot) * scale
        # |error of an element of P|: its bf16 rounding, and what the logits' error makes of p
        ep = abs(scale) * ((p - hot).abs() * 2.0 ** -8 * 1.01 + p * (2 * dl[:, None] + 2.0 ** -20))
        for name, out, ref, err, k, terms in (
                ("d_hidden", self.dh, d @ w, ep @ w.abs(), self.V, d.abs() @ w.abs()),
                ("d_weight", self.dw, d.t() @ h, ep.t() @ h.abs(), n, d.abs().t() @ h.abs())):
            if out is None:
                continue
            if name == "d_hidden":
                assert bool((out[away] == 0).all())
                out = out[keep]
            tol = 1.01 * err + (k / 16 + 40) * 2.0 ** -22 * terms + 2.0 ** -8 * 1.01 * ref.abs() + 1e-36
            off = (out.double() - ref).abs()
            assert bool((off <= tol).all()), (name, float((off / tol).max()))
        return self


SIZES = [(1, 1, 1), (1, 32003, 96), (2, 2, 7), (3, 257, 8), (31, 255, 63), (33, 256, 64), (50, 128, 64), (127, 1000, 65),
         (128, 513, 129), (129, 40, 2050), (255, 130, 72), (256, 256, 256), (257, 777, 200), (513, 1025, 40),
         (1021, 5003, 301), (2100, 32003, 64)]


@gpu
@pytest.mark.parametrize("T,V,D", SIZES)
def test_sizes(ss, T, V, D):
    Case(T, V, D, seed=T).run(ss).check()


@gpu
@pytest.mark.parametrize("mask", ["all", "all_but_last", "alternate", "first_half", "random"])
@pytest.mark.parametrize("T,V,D", [(1, 50, 16), (64, 300, 64), (65, 300, 64), (300, 700, 100), (700, 513, 264)])
def test_masks(ss, T, V, D, mask):
    """Ignored tokens whose rows hold NaN and infinities leave nothing anywhere."""
    c = Case(T, V, D, mask=mask, seed=3)
    away = c.y == c.ignore
    c.h[away] = float("nan")
    if int(away.sum()) > 1:
        c.h[torch.nonzero(away)[1, 0]] = float("inf")
    c.run(ss).check()
    if mask == "all":
        assert float(c.loss) == 0.0 and bool((c.dw == 0).all()) and bool((c.dh == 0).all())


@gpu
def test_no_tokens(ss):
    c = Case(0, 70, 24).run(ss)
    assert float(c.loss) == 0.0 and bool((c.dw == 0).all())


@gpu
@pytest.mark.parametrize("ignore", [0, 7, -1])
def test_ignore_index(ss, ignore):
    Case(200, 90, 48, mask="random", ignore=ignore).run(ss).check()


@gpu
@pytest.mark.parametrize("h_extra,w_extra,offset,out_extra,out_offset", [
    (8, 8, 0, 8, 0), (5, 0, 0, 0, 0), (0, 5, 0, 3, 0), (0, 0, 3, 0, 1), (1, 7, 1, 1, 7), (16, 24, 8, 5, 4)])
@pytest.mark.parametrize("D", [64, 61])
def test_strides(ss, D, h_extra, w_extra, offset, out_extra, out_offset):
    """Rows at any stride and offset; nothing is written between the outputs' rows."""
    c = Case(150, 300, D, mask="random", h_extra=h_extra, w_extra=w_extra, offset=offset)
    c.run(ss, out_extra=out_extra, out_offset=out_offset).check()
    assert int((c.dhbuf == 5.0).sum()) >= c.dhbuf.numel() - 150 * D
    c.dh.zero_(), c.dw.zero_()
    assert int((c.dhbuf == 5.0).sum()) == c.dhbuf.numel() - 150 * D
    assert int((c.dwbuf == 5.0).sum()) == c.dwbuf.numel() - 300 * D


@gpu
@pytest.mark.parametrize("dh,dw", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("reduction,grad_scale", [("mean", 1.0), ("sum", 0.25), ("mean", -512.0)])
def test_outputs_and_scales(ss, dh, dw, reduction, grad_scale):
    c = Case(300, 600, 80, mask="random")
    c.run(ss, dh=dh, dw=dw, reduction=reduction, grad_scale=grad_scale).check(reduction, grad_scale)


@gpu
def test_pieces(ss):
    """More than one piece of the vocabulary, the last one short, and tokens that leave whole tiles empty."""
    Case(2304, 60001, 72, mask="random", seed=5).run(ss).check()


@gpu
@pytest.mark.parametrize("T", [16384, 20001])
@pytest.mark.parametrize("mask", ["none", "random", "first_half"])
def test_many_tokens(ss, T, mask):
    """So many tokens that those that count are counted by chunks first."""
    Case(T, 130, 24, mask=mask, seed=6).run(ss).check()


@gpu
@pytest.mark.parametrize("std", [1e-3, 8.0])
def test_flat_and_peaked(ss, std):
    """Nearly equal logits, and logits that put all the mass on one class (exponentials that underflow)."""
    Case(130, 900, 128, std=std).run(ss).check()


@gpu
def test_target_out_of_range(ss):
    c = Case(40, 30, 16)
    c.y[7] = 30
    c.run(ss)
    assert math.isnan(float(c.token_loss[7])) and math.isnan(float(c.loss))
    rest = torch.ones(40, dtype=torch.bool, device="cuda")
    rest[7] = False
    assert bool(c.token_loss[rest].isfinite().all())


@gpu
def test_nan_comes_through(ss):
    c = Case(40, 30, 16)
    c.h[5, 3] = float("nan")
    c.run(ss)
    assert math.isnan(float(c.token_loss[5])) and math.isnan(float(c.loss))
    assert bool(c.token_loss[:5].isfinite().all())
    assert bool(c.dh[5].isnan().all()) and bool(c.dh[:5].isfinite().all())


@gpu
@pytest.mark.parametrize("T,V,grad", [(1, 12003, False), (2, 12003, False), (2, 12003, True), (3, 20001, False),
                                      (4, 20001, True), (40, 100, True), (40, 100, False), (300, 700, False),
                                      (300, 700, True), (70, 3001, True)])
@pytest.mark.parametrize("rows", ["pair", "four", "first_32", "second_half", "beside_the_target", "with_minus_infinities"])
def test_nan_weight_rows_come_through(ss, T, V, grad, rows):
    """A NaN in the head's weight makes every logit of its class NaN, and with it every token's loss (the definition's
    sum holds that logit), wherever the class lies among those summed together and whatever follows it."""
    c = Case(T, V, 72, seed=8)
    c.y[:] = V - 2  # not one of the rows that are NaN
    low, high = {"pair": (0, 2), "four": (0, 4), "first_32": (0, 32), "second_half": (128 % (V - 40), 128 % (V - 40) + 32),
                 "beside_the_target": (6, 7), "with_minus_infinities": (0, 32)}[rows]
    if rows == "beside_the_target":
        c.y[:] = 7
    if rows == "with_minus_infinities":
        c.h.abs_()
        c.w[low:high] = -math.inf
        c.w[low + 1] = math.nan
    else:
        c.w[low:high] = math.nan
    c.run(ss, dh=grad, dw=grad)
    assert math.isnan(float(c.loss)) and bool(c.token_loss.isnan().all())
    if grad:
        assert bool(c.dh.isnan().all()) and bool(c.dw.isnan().all())


FORMS = [(1, 500, False), (2, 500, True), (4, 500, False), (4, 500, True), (40, 100, True), (40, 100, False),
         (300, 700, False), (300, 700, True)]


@gpu
@pytest.mark.parametrize("T,V,grad", FORMS)
def test_infinite_target_logit(ss, T, V, grad):
    """A logit of +inf, here the target's own: its loss is inf - inf."""
    c = Case(T, V, 72, seed=9)
    c.h.abs_()
    c.y[:] = 11
    c.w[11] = math.inf
    c.run(ss, dh=grad, dw=grad)
    assert math.isnan(float(c.loss)) and bool(c.token_loss.isnan().all())
    if grad:
        assert bool(c.dh.isnan().all()) and bool(c.dw.isnan().all())


@gpu
@pytest.mark.parametrize("T,V,grad", FORMS)
def test_target_logit_of_minus_infinity(ss, T, V, grad):
    """A class whose logits are -inf is no part of any sum; where it is the target, the loss is infinite and P is the
    other classes' softmax with -1 in its place."""
    c = Case(T, V, 72, seed=9)
    c.h.abs_()
    c.y[c.y == 11] = 12
    c.y[::2] = 11
    c.w[11] = -math.inf
    c.run(ss, dh=grad, dw=grad)
    assert float(c.loss) == math.inf and bool((c.token_loss[::2] == math.inf).all())
    h, w = c.h.double(), c.w.double()
    w[11] = 0.0
    logits = h @ w.t()
    logits[:, 11] = -math.inf
    want = torch.logsumexp(logits, 1) - logits.gather(1, c.y[:, None]).squeeze(1)
    # dl as above: (72 / 16 + 2) * 2^-22 of a sum below 1000
    assert bool(((c.token_loss[1::2].double() - want[1::2]).abs() <= 2e-3).all())
    if grad:
        p = torch.softmax(logits, 1)
        p = (p - torch.nn.functional.one_hot(c.y, V)) / T
        # two roundings to bf16, 2^-8 each, and 2e-3 of a p for its logit
        assert bool(((c.dw.double() - p.t() @ h).abs() <= 0.012 * (p.abs().t() @ h) + 1e-36).all())


@gpu
@pytest.mark.parametrize("T,grad", [(1, False), (2, True), (4, True), (40, True), (40, False), (300, True)])
def test_no_finite_logit(ss, T, grad):
    """Every logit -inf, or the only class's NaN: no loss is defined.  A lone finite class has a loss of 0."""
    for V, value in ((1, math.nan), (1, -math.inf), (70, -math.inf)):
        c = Case(T, V, 72, seed=10)
        c.h.abs_()
        c.w[:] = value
        c.run(ss, dh=grad, dw=grad)
        assert math.isnan(float(c.loss)) and bool(c.token_loss.isnan().all()), (V, value)
        if grad:
            assert bool(c.dh.isnan().all()) and bool(c.dw.isnan().all()), (V, value)
    c = Case(T, 1, 72, seed=10).run(ss, dh=grad, dw=grad)
    assert float(c.loss) == 0.0 and bool((c.token_loss == 0).all())
    if grad:
        assert bool((c.dh == 0).all()) and bool((c.dw == 0).all())


@gpu
@pytest.mark.parametrize("T,grad", [(1, False), (2, True), (3, False), (4, False), (4, True), (30, True), (150, False),
                                    (150, True)])
@pytest.mark.parametrize("D,extra", [(24, 0), (20, 4), (72, 0), (61, 3), (61, 0)])
def test_nothing_beside_the_rows_is_read(ss, T, grad, D, extra):
    """NaN between the rows and around the tensors, with rows on 16-byte boundaries and off."""
    c = Case(T, 300, D, h_extra=extra, w_extra=extra)
    for view, buf in ((c.h, c.hbuf), (c.w, c.wbuf)):
        keep = view.clone()
        buf.fill_(float("nan"))
        view.copy_(keep)
    c.run(ss, dh=grad, dw=grad).check()


def dominant_channel(ss, D, at):
    """Mean signed error, relative to the logit, of log-sum-exps that hang on one logit of about 37, which a single
    channel of the hidden states makes and the others add noise to."""
    T, V = 1024, 64
    gen = torch.Generator("cuda").manual_seed(12 + at)
    h = torch.randn(T, D, generator=gen, device="cuda") * 0.1
    h[:, at] = 20 + torch.randn(T, generator=gen, device="cuda")
    w = torch.randn(V, D, generator=gen, device="cuda") * (0.01 / math.sqrt(D))
    w[0] = torch.randn(D, generator=gen, device="cuda") * 0.02
    w[0, at] = 37 / 20
    h, w, y = h.to(BF), w.to(BF), torch.ones(T, dtype=torch.int64, device="cuda")
    loss, tl = torch.empty(1, device="cuda"), torch.empty(T, device="cuda")
    ws = torch.empty(ss.ss_linear_ce_workspace(T, D, V, False), dtype=torch.uint8, device="cuda")
    ss.ss_linear_cross_entropy(h, w, y, loss, ws, token_loss_out=tl)
    logits = h.double() @ w.double().t()
    want = torch.logsumexp(logits, 1) - logits[:, 1]
    return float(((tl.double() - want) / logits[:, 0]).mean())


# What the accumulator drops, and what is made good of it.  An add drops what lies below the running sum's 24 bits, half
# a unit of the last place on average: 2^-25 to 2^-24 of the sum, for each 16 products behind the dominant one.  1.55e-8
# (just above 2^-26) of each 16 products is added back, up to 16384 of them.  2^-22: the fp32 roundings beside it.

@gpu
def test_dropped_bits_over_the_positions(ss):
    """A channel at any place: half of the adds come behind it on average, which leaves 2^-26 to 2^-25 less 1.55e-8."""
    D = 4096
    mean = sum(dominant_channel(ss, D, at) for at in range(D // 32, D, D // 16)) / 16
    assert abs(mean) <= D / 16 * 2.0 ** -26 + 2.0 ** -22


@gpu
@pytest.mark.parametrize("D", [4096, 16384, 65536])
def test_dropped_bits_first_and_last(ss, D):
    """A channel at the start, behind which every add drops something, and at the end, where what is added back is the
    whole error."""
    back = 1.55e-8 * min(D, 16384) / 16
    assert abs(dominant_channel(ss, D, 3)) <= D / 16 * 2.0 ** -24 + 2.0 ** -22
    assert abs(dominant_channel(ss, D, D - 5)) <= back + 2.0 ** -22


@gpu
def test_same_bits_twice_and_on_another_stream(ss):
    c = Case(700, 3001, 136, mask="random")
    c.run(ss)
    first = [c.loss.clone(), c.token_loss.clone(), c.dh.clone(), c.dw.clone()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c.run(ss)
    side.synchronize()
    for a, b in zip(first, (c.loss, c.token_loss, c.dh, c.dw)):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("T,V,D", [(3, 700, 72), (50, 128, 64), (300, 700, 100)])
def test_captured(ss, T, V, D):
    """A captured call (of each form) replays on what the inputs hold by then."""
    c, other = Case(T, V, D, seed=1), Case(T, V, D, seed=2, mask="random")
    c.run(ss)
    stream = torch.cuda.Stream()
    ws = torch.empty(ss.ss_linear_ce_workspace(T, D, V, True, stage_weight=True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ss.ss_linear_cross_entropy(c.h, c.w, c.y, c.loss, ws, token_loss_out=c.token_loss, d_hidden=c.dh,
                                   d_weight=c.dw, stream=stream)
    for a, b in ((c.h, other.h), (c.w, other.w), (c.y, other.y)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    c.check()


@gpu
@pytest.mark.parametrize("T,grad,launch,reduction", [(300, False, 0, "mean"), (20, False, 0, "sum"), (300, True, 0, "mean"),
                                                     (300, True, 1, "sum"), (300, True, 2, "mean"), (3, True, 1, "mean")])
def test_a_wait_that_runs_out(ss, T, grad, launch, reduction):
    """One wait that nothing ends gives up by itself: the loss says so, the device stays usable, the next call is right."""
    c = Case(T, 3000, 136, mask="random" if T > 3 else "none", seed=11)
    ss.ss_linear_ce_expire_wait(launch)
    c.run(ss, dh=grad, dw=grad, reduction=reduction)
    assert math.isnan(float(c.loss))
    away = c.y == c.ignore
    assert bool((c.token_loss[away] == 0).all())
    if launch == 0:
        assert bool(c.token_loss[~away].isnan().all())
        if grad:
            assert bool(c.dh[~away].isnan().all()) and bool(c.dw.isnan().all())
    c.run(ss, dh=grad, dw=grad, reduction=reduction).check(reduction)


@gpu
def test_workspace_used_again(ss):
    """Another call's leftovers in the workspace change nothing."""
    big, small = Case(600, 2000, 136, seed=1), Case(90, 700, 100, mask="random", seed=2)
    n = max(ss.ss_linear_ce_workspace(c.T, c.D, c.V, True) for c in (big, small))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    big.run(ss, workspace=ws).check()
    small.run(ss, workspace=ws).check()
    big.run(ss, workspace=ws).check()


@gpu
def test_offsets_past_32_bits(ss):
    """A weight of more than 2^31 elements: the last rows' logits and gradients land where they belong."""
    T, V, D = 3, (1 << 31) // 1024 + 4099, 1024
    w = torch.zeros(V, D, dtype=BF, device="cuda")
    gen = torch.Generator("cuda").manual_seed(1)
    rows = torch.tensor([0, 1, V // 2, V - 2, V - 1], device="cuda")
    w[rows] = torch.randn(5, D, generator=gen, device="cuda").to(BF)
    h = torch.randn(T, D, generator=gen, device="cuda").to(BF)
    y = rows[[4, 0, 3]].clone()
    dw = torch.full((V, D), 5.0, dtype=BF, device="cuda")
    dh = torch.empty(T, D, dtype=BF, device="cuda")
    loss, tl = torch.empty(1, device="cuda"), torch.empty(T, device="cuda")
    ws = torch.empty(ss.ss_linear_ce_workspace(T, D, V, True), dtype=torch.uint8, device="cuda")
    ss.ss_linear_cross_entropy(h, w, y, loss, ws, token_loss_out=tl, d_hidden=dh, d_weight=dw)
    wr, hd = w[rows].double(), h.double()
    lr = hd @ wr.t()
    lse = torch.log((V - 5) + lr.exp().sum(1))  # every other logit is 0
    hit = lr[torch.arange(3), torch.tensor([4, 0, 3], device="cuda")]
    # dl as above with sum |h w| below 1024; 2^21 exponentials summed in fp32 by 8 threads a row
    assert bool(((tl.double() - (lse - hit)).abs() <= 1e-3).all())
    p = (lr - lse[:, None]).exp() / 3
    p[torch.arange(3), torch.tensor([4, 0, 3], device="cuda")] -= 1 / 3
    want = p.t() @ hd
    tol = 0.01 * (p.abs().t() @ hd.abs()) + 1e-30
    assert bool(((dw[rows].double() - want).abs() <= tol).all())
    rest = (-lse).exp() @ hd / 3  # of a row whose logits are all 0
    tol = 0.01 * ((-lse).exp() @ hd.abs() / 3)
    for v in (2, 12345, V // 2 + 1, (1 << 31) // 1024 + 1, V - 3):
        assert bool(((dw[v].double() - rest).abs() <= tol).all()), v
    want = p @ wr
    assert bool(((dh.double() - want).abs() <= 0.01 * (p.abs() @ wr.abs()) + 1e-30).all())


@gpu
def test_gradient_against_differences(ss):
    """<d_weight, d> against the loss at weight +- e d, both exactly bf16: the difference quotient is off by at most
    e^2 / 6 times the third derivative, a third central moment of the direction's logits, (2 max |<h, d>|)^3."""
    T, V, D, e = 40, 60, 24, 2.0 ** -5
    gen = torch.Generator("cuda").manual_seed(4)
    h = (torch.randint(-8, 9, (T, D), generator=gen, device="cuda") / 16).to(BF)
    w = (torch.randint(-16, 17, (V, D), generator=gen, device="cuda") / 32).to(BF)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    ws = torch.empty(ss.ss_linear_ce_workspace(T, D, V, True), dtype=torch.uint8, device="cuda")
    loss = torch.empty(1, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ss.ss_linear_cross_entropy(h, w, y, loss, ws, d_hidden=dh, d_weight=dw)

    def value(h, w):
        ss.ss_linear_cross_entropy(h, w, y, loss, ws)
        return float(loss)

    for k in range(4):
        d = (torch.randint(0, 2, (V, D), generator=gen, device="cuda") * 2 - 1).to(BF)
        quotient = (value(h, w + e * d) - value(h, w - e * d)) / (2 * e)
        moment = (2 * float((h.double() @ d.double().t()).abs().max())) ** 3
        rounding = 2.0 ** -8 * float((dw.double() * d.double()).abs().sum()) + 1e-6 / e
        assert abs(float((dw.double() * d.double()).sum()) - quotient) <= e * e / 6 * moment + rounding
        d = (torch.randint(0, 2, (T, D), generator=gen, device="cuda") * 2 - 1).to(BF)
        quotient = (value(h + e * d, w) - value(h - e * d, w)) / (2 * e)
        moment = (2 * float((d.double() @ w.double().t()).abs().max())) ** 3
        rounding = 2.0 ** -8 * float((dh.double() * d.double()).abs().sum()) + 1e-6 / e
        assert abs(float((dh.double() * d.double()).sum()) - quotient) <= e * e / 6 * moment + rounding


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_refusals_on_the_host(ss):
    import ctypes
    lib = ss.lib()
    n = ctypes.c_size_t()
    size = lambda *a: lib.ss_linear_ce_workspace(*a, ctypes.byref(n))
    assert size(4, 64, 100, 0) == ss.SS_OK and n.value > 0
    plain = n.value
    assert size(4, 64, 100, ss.SS_CE_GRADIENT) == ss.SS_OK and n.value > plain
    assert size(4, 64, 100, ss.SS_CE_STAGE_WEIGHT) == ss.SS_OK and n.value >= plain + 100 * 64 * 2
    assert size(-1, 64, 100, 0) == ss.SS_EINVAL
    assert size(4, 0, 100, 0) == ss.SS_EINVAL
    assert size(4, 64, 0, 0) == ss.SS_EINVAL
    assert size(4, 64, 100, 8) == ss.SS_EINVAL
    assert size(1 << 40, 64, 100, 0) == ss.SS_EOVERFLOW
    assert lib.ss_linear_ce_workspace(4, 64, 100, 0, None) == ss.SS_EINVAL
    at = 1 << 20  # an address that is never touched
    good = dict(num_tokens=4, hidden_size=64, vocab_size=100, hidden=at, hidden_stride=64, weight=at, weight_stride=64,
                targets=at, ignore_index=-100, reduction=0, grad_scale=1.0, loss_out=at, token_loss_out=None,
                d_hidden=None, d_hidden_stride=0, d_weight=None, d_weight_stride=0, workspace=at, workspace_bytes=1 << 30)

    def call(**kw):
        a = ss._LinearCE(*{**good, **kw}.values())
        return lib.ss_linear_cross_entropy(ctypes.byref(a), None)

    assert lib.ss_linear_cross_entropy(None, None) == ss.SS_EINVAL
    for kw in (dict(num_tokens=-1), dict(hidden_size=0), dict(vocab_size=0), dict(hidden=None), dict(weight=None),
               dict(targets=None), dict(loss_out=None), dict(workspace=None), dict(workspace_bytes=16),
               dict(hidden_stride=63), dict(weight_stride=8), dict(reduction=2), dict(grad_scale=math.nan),
               dict(grad_scale=math.inf), dict(d_hidden=at, d_hidden_stride=1), dict(d_weight=at, d_weight_stride=63)):
        assert call(**kw) == ss.SS_EINVAL, kw
    for kw in (dict(hidden=at + 1), dict(weight=at + 1), dict(targets=at + 4), dict(loss_out=at + 2),
               dict(token_loss_out=at + 1), dict(workspace=at + 16), dict(d_hidden=at + 1, d_hidden_stride=64),
               dict(d_weight=at + 1, d_weight_stride=64)):
        assert call(**kw) == ss.SS_EALIGN, kw
    for kw in (dict(num_tokens=1 << 40), dict(vocab_size=1 << 30), dict(weight_stride=1 << 60),
               dict(hidden_stride=1 << 62)):
        assert call(**kw) == ss.SS_EOVERFLOW, kw


def test_expired_wait_is_for_one_launch(ss):
    with pytest.raises(ss.ShardStateError) as e:
        ss.ss_linear_ce_expire_wait(-2)
    assert e.value.status == ss.SS_EINVAL
    ss.ss_linear_ce_expire_wait(-1)


def test_scales_beyond_fp32_are_refused(ss):
    """A finite scale that fp32 rounds to infinity would turn gradients of 0 to NaN."""
    import ctypes
    at = 1 << 20  # an address that is never touched: the workspace's is refused next
    for scale, want in ((3.5e38, ss.SS_EINVAL), (-1e300, ss.SS_EINVAL), (3.4e38, ss.SS_EALIGN)):
        a = ss._LinearCE(4, 64, 100, at, 64, at, 64, at, -100, 0, scale, at, None, at, 64, at, 64, at + 16, 1 << 30)
        assert ss.lib().ss_linear_cross_entropy(ctypes.byref(a), None) == want


@gpu
def test_refusals_of_the_binding(ss):
    c = Case(10, 20, 16)
    launched = ss.ss_launch_count()  # of refused calls: none
    loss = torch.empty(1, device="cuda")
    ws = torch.empty(ss.ss_linear_ce_workspace(10, 16, 20, True), dtype=torch.uint8, device="cuda")
    for kw in (dict(hidden=c.h.cpu()), dict(targets=c.y.cpu()), dict(loss_out=loss.cpu()), dict(workspace=ws.cpu()),
               dict(hidden=c.h.float()), dict(hidden=c.h[0]), dict(weight=c.w.t()), dict(targets=c.y.int()),
               dict(targets=c.y[:9]), dict(loss_out=loss.double()), dict(reduction="none"), dict(d_hidden=c.w),
               dict(d_weight=c.h), dict(token_loss_out=torch.empty(9, device="cuda")), dict(workspace=ws[:256])):
        with pytest.raises(ss.ShardStateError) as e:
            ss.ss_linear_cross_entropy(**{**dict(hidden=c.h, weight=c.w, targets=c.y, loss_out=loss, workspace=ws), **kw})
        assert e.value.status == ss.SS_EINVAL
    assert ss.ss_launch_count() == launched
