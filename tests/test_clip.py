"""The gradient norm, clipping, and the sharded step with clipping, against the
formulas in 64 bits.

Tolerances.  A CTA's sum of squares is fp32: 32 squares in a thread and 8 adds
across the CTA, every term non-negative, so its relative error is at most
40 * 2^-24 = 2.4e-6; the sum of the CTAs is fp64.  The norm is its root, rounded
to fp32: half of that and 2^-24, below 1.3e-6; the factor the same and another
rounding.  NORM_RTOL = 2e-6 covers both.  What is scaled is compared bit for bit
with the product of the input and the factor the GPU reported, rounded once.
"""
import math

import numpy as np
import pytest
import torch

import workloads as W
from tests.helpers import check_adamw_state

NORM_RTOL = 2e-6
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import __graft_entry__
    __graft_entry__.build()
    import sharded_state_gb300 as ss
    return ss


def workspace(ss):
    return torch.empty(ss.SS_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def tensors(sizes, dtypes, offsets, seed=0, std=1e-2):
    """Contiguous tensors, tensor k starting offsets[k] elements past a 16-byte boundary,
    between sentinel elements."""
    gen = torch.Generator("cuda").manual_seed(seed)
    out, whole = [], []
    for n, dt, o in zip(sizes, dtypes, offsets):
        buf = torch.full((n + 64,), 7.0, dtype=dt, device="cuda")
        buf[16 + o:16 + o + n] = torch.randn(n, generator=gen, device="cuda") * std
        out.append(buf[16 + o:16 + o + n])
        whole.append(buf)
    return out, whole


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


BF, F32 = torch.bfloat16, torch.float32
LISTS = {
    "one_element": ([1], [BF], [0]),
    "empty_list": ([], [], []),
    "only_empties": ([0, 0], [BF, F32], [0, 1]),
    "tiny_mlp": ([8192, 128, 8192, 64, 64], [BF] * 5, [0] * 5),
    "odd_offsets": ([1, 7, 8, 9, 15, 16, 17, 0, 100, 8191, 8192, 8193], [BF] * 12, [1, 2, 3, 4, 5, 6, 7, 1, 3, 1, 0, 7]),
    "fp32_offsets": ([1, 3, 4, 5, 4095, 4096, 4097, 20000], [F32] * 8, [1, 2, 3, 1, 2, 3, 0, 1]),
    "mixed": ([33, 70000, 5, 12345, 999], [BF, F32, F32, BF, BF], [3, 1, 2, 5, 0]),
    "many": ([(i * 37) % 300 for i in range(1300)], [BF if i % 3 else F32 for i in range(1300)],
             [i % (8 if i % 3 else 4) for i in range(1300)]),
    "large": ([30_000_001, 9_999_999], [BF, F32], [3, 1]),
}


@gpu
@pytest.mark.parametrize("name", LISTS)
def test_grad_norm(ss, name):
    ts, _ = tensors(*LISTS[name])
    norm = torch.full((2,), -1.0, device="cuda")
    ss.ss_grad_norm(ts, norm, workspace(ss))
    want = norm64(ts)
    assert float(norm[1]) == 1.0
    assert abs(float(norm[0]) - want) <= NORM_RTOL * want
    again = torch.empty(2, device="cuda")
    ss.ss_grad_norm(ts, again, workspace(ss))
    assert torch.equal(norm, again)


@gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("clips", [True, False])
@pytest.mark.parametrize("name", LISTS)
def test_clip_grads(ss, name, clips, in_place):
    sizes, dtypes, offsets = LISTS[name]
    ts, whole = tensors(sizes, dtypes, offsets)
    was = [t.clone() for t in ts]
    want = norm64(ts)
    max_norm = want * (0.37 if clips else 3.0) + (0.0 if clips else 1.0)
    # outputs at other offsets than the inputs
    outs, owhole = (ts, whole) if in_place else tensors(
        sizes, dtypes, [(o * 5 + 3) % (8 if d == BF else 4) for o, d in zip(offsets, dtypes)], std=0.0)
    norm = torch.empty(2, device="cuda")
    ss.ss_clip_grads(ts, max_norm, norm, workspace(ss), out=None if in_place else outs)
    n, c = (float(x) for x in norm)
    assert abs(n - want) <= NORM_RTOL * want
    c64 = min(1.0, max_norm / (want + 1e-6))
    assert abs(c - c64) <= NORM_RTOL * c64
    if not clips:
        assert c == 1.0
    for x, o, buf, d in zip(was, outs, owhole, dtypes):
        assert torch.equal(o, (x.float() * c).to(d))
        assert int((buf == 7.0).sum()) == buf.numel() - o.numel()  # nothing beside it was written
    if not in_place:
        for x, t in zip(was, ts):
            assert torch.equal(x, t)


@gpu
@pytest.mark.parametrize("bad,norm_is,factor_is", [(math.nan, math.nan, math.nan), (math.inf, math.inf, 0.0),
                                                   (-math.inf, math.inf, 0.0), (3e38, math.inf, 0.0)])
def test_not_finite(ss, bad, norm_is, factor_is):
    ts, _ = tensors([1000, 77], [F32, BF], [1, 3])
    ts[0][512] = bad
    norm = torch.empty(2, device="cuda")
    ss.ss_clip_grads(ts, 1.0, norm, workspace(ss))
    same = lambda a, b: a == b or (math.isnan(a) and math.isnan(b))
    assert same(float(norm[0]), norm_is) and same(float(norm[1]), factor_is)
    rest = torch.cat([ts[0][:512].float(), ts[1].float()])
    assert bool(rest.isnan().all()) if math.isnan(factor_is) else bool((rest == 0).all())
    if math.isinf(bad):
        assert math.isnan(float(ts[0][512]))  # inf * 0


FORM_LISTS = {"cluster": [1000, 77], "cooperative": [300_000, 77], "two_launches": [30_000_001, 77]}


@gpu
@pytest.mark.parametrize("bad", [math.inf, 3e38])
@pytest.mark.parametrize("form", FORM_LISTS)
def test_unlimited_with_an_infinite_norm(ss, form, bad):
    """max_norm = +inf never clips: an infinite norm leaves every element as it is."""
    ts, _ = tensors(FORM_LISTS[form], [F32, BF], [1, 3])
    ts[0][512] = bad
    was = [t.clone() for t in ts]
    outs = [torch.empty_like(t) for t in ts]
    norm = torch.empty(2, device="cuda")
    ss.ss_clip_grads(ts, math.inf, norm, workspace(ss), out=outs)
    assert norm.tolist() == [math.inf, 1.0]
    for x, o in zip(was, outs):
        assert torch.equal(x, o)
    ss.ss_clip_grads(ts, math.inf, norm, workspace(ss))
    for x, t in zip(was, ts):
        assert torch.equal(x, t)
    ts[0][512] = math.nan
    ss.ss_clip_grads(ts, math.inf, norm, workspace(ss))
    assert bool(norm.isnan().all()) and bool(ts[1].isnan().all())


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, 3e38])
@pytest.mark.parametrize("form", FORM_LISTS)
def test_norm_alone_not_finite(ss, form, bad):
    """The norm alone has a factor of 1, whatever the norm."""
    ts, _ = tensors(FORM_LISTS[form], [F32, BF], [1, 3])
    ts[0][512] = bad
    norm = torch.empty(2, device="cuda")
    ss.ss_grad_norm(ts, norm, workspace(ss))
    assert float(norm[1]) == 1.0
    assert math.isnan(float(norm[0])) if math.isnan(bad) else float(norm[0]) == math.inf


@gpu
def test_zero_and_unlimited(ss):
    ts, _ = tensors([500], [BF], [1])
    was = ts[0].clone()
    norm = torch.empty(2, device="cuda")
    ss.ss_clip_grads(ts, math.inf, norm, workspace(ss))
    assert float(norm[1]) == 1.0 and torch.equal(ts[0], was)
    ss.ss_clip_grads(ts, 0.0, norm, workspace(ss))
    assert float(norm[1]) == 0.0 and bool((ts[0] == 0).all())
    ss.ss_clip_grads(ts, 1.0, norm, workspace(ss))  # all zero: norm 0, nothing to clip
    assert norm.tolist() == [0.0, 1.0]


@gpu
def test_handle_and_stream(ss):
    """The marshalled call, on a stream of its own, twice with other gradients in the same place."""
    ts, _ = tensors([4000, 4001], [BF, F32], [0, 1])
    outs = [torch.empty_like(t) for t in ts]
    norm = torch.empty(2, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    clip = ss.GradClip(ts, 0.1, norm, workspace(ss), out=outs)
    with torch.cuda.stream(side):
        for k in range(2):
            for t in ts:
                t.mul_(1 + k)
            clip()
            side.synchronize()
            assert abs(float(norm[0]) - norm64(ts)) <= NORM_RTOL * norm64(ts)
            for t, o in zip(ts, outs):
                assert torch.equal(o, (t.float() * norm[1]).to(t.dtype))


@gpu
@pytest.mark.parametrize("name", ["tiny_mlp", "mixed", "large"])
def test_captured(ss, name):
    """A captured call replays on what the tensors hold by then."""
    ts, _ = tensors(*LISTS[name])
    outs = [torch.empty_like(t) for t in ts]
    norm, ws = torch.empty(2, device="cuda"), workspace(ss)
    stream = torch.cuda.Stream()
    clip = ss.GradClip(ts, 0.1, norm, ws, out=outs, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        clip()
    for t in ts:
        t.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm[0]) - norm64(ts)) <= NORM_RTOL * norm64(ts)
    for t, o in zip(ts, outs):
        assert torch.equal(o, (t.float() * norm[1]).to(t.dtype))


# Forms that only larger or longer lists take: more than 8192 partials, with a fold launch of their own; more than 256
# tensors with at most 1024 partials, which the second pass folds itself.
LONG_LISTS = {
    "fold_launch": ([70_000_001, 9_999, 600_001], [BF, F32, F32], [5, 1, 3]),
    "self_folding": ([(i * 37) % 300 + 1 for i in range(400)], [BF if i % 3 else F32 for i in range(400)],
                     [i % (8 if i % 3 else 4) for i in range(400)]),
}


@gpu
@pytest.mark.parametrize("name", LONG_LISTS)
def test_grad_norm_of_long_lists(ss, name, monkeypatch):
    monkeypatch.setitem(LISTS, name, LONG_LISTS[name])
    test_grad_norm(ss, name)


@gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("clips", [True, False])
@pytest.mark.parametrize("name", LONG_LISTS)
def test_clip_long_lists(ss, name, clips, in_place, monkeypatch):
    monkeypatch.setitem(LISTS, name, LONG_LISTS[name])
    test_clip_grads(ss, name, clips, in_place)


# Above about 17 GB a partial is a sum of 64 values a thread: 72 * 2^-24 of it at most, half of that in the norm, and 2^-24.
HUGE_RTOL = 2.3e-6


def repeated(n, dtype):
    """n elements of a random block of 2^26 again and again, and the sum of their squares."""
    gen = torch.Generator("cuda").manual_seed(7)
    block = (torch.randn(1 << 26, generator=gen, device="cuda") * 1e-2).to(dtype)
    out = torch.empty(n, dtype=dtype, device="cuda")
    for a in range(0, n, 1 << 26):
        out[a:a + (1 << 26)] = block[:min(1 << 26, n - a)]
    sq = lambda x: float(x.double().square().sum())
    return out, block, n // (1 << 26) * sq(block) + sq(block[:n % (1 << 26)])


@gpu
def test_clip_more_than_the_partials_hold(ss):
    """So much that a CTA takes more than one round of tiles: the norm, and clipping in place."""
    n = 8_700_000_003
    buf, block, sq = repeated(n, BF)
    ts = [buf[:5_000_000_001], buf[5_000_000_001:]]  # the second starts 2 bytes past a boundary
    norm, ws = torch.empty(2, device="cuda"), workspace(ss)
    ss.ss_grad_norm(ts, norm, ws)
    want = math.sqrt(sq)
    assert abs(float(norm[0]) - want) <= HUGE_RTOL * want and float(norm[1]) == 1.0
    ss.ss_clip_grads(ts, 0.25 * want, norm, ws)
    c = float(norm[1])
    assert abs(float(norm[0]) - want) <= HUGE_RTOL * want and abs(c - 0.25) <= HUGE_RTOL
    scaled = (block.float() * c).to(BF)
    for a in range(0, n, 1 << 26):
        assert torch.equal(buf[a:a + (1 << 26)], scaled[:min(1 << 26, n - a)]), a


# ---------------------------------------------------------------------------
# the sharded step
# ---------------------------------------------------------------------------

def plan_of(ss, kind):
    """Name -> (ParamSet, groups called one by one)."""
    return {
        "tiny": W.tiny_mlp(2),
        "per_param_3": W.awkward_2d(3, count=40, max_rows=500),
        "flat_false_7": W.awkward_1d(7, W.FLAT_ORIG_FALSE, BF, count=60, max_len=3000),
        "flat_true_5_fp32": W.awkward_1d(5, W.FLAT_ORIG_TRUE, F32, count=60, max_len=3000),
        "one_rank": W.tiny_mlp(1, W.FLAT_ORIG_FALSE),
        "flat_12": W.awkward_1d(12, W.FLAT_ORIG_FALSE, BF, count=30, max_len=1000),
        "flat_17_fp32": W.awkward_1d(17, W.FLAT_ORIG_TRUE, F32, count=30, max_len=1000),
        "groups": W.llama_1b2(4, layers=2, hidden=64, ffn=100, vocab=130),
        # groups whose ranges start and end inside a 16-byte vector, and an empty one
        "tiny_groups": W.ParamSet([f"p{i}" for i in range(7)], [(1,), (3,), (0,), (5,), (9,), (2,), (30,)],
                                  [1, 1, 1, 1, 1, 1, 1], 3, W.PER_PARAM_DIM0, BF, seed=9),
    }[kind]


KINDS = ["tiny", "per_param_3", "flat_false_7", "flat_true_5_fp32", "one_rank", "flat_12", "flat_17_fp32", "groups",
         "tiny_groups"]


class Sharded:
    def __init__(self, ss, kind, with_master=True):
        self.ss, self.ps = ss, plan_of(ss, kind)
        d0, inner = self.ps.dim0_inner()
        self.plan = ss.fsdp_plan_create(self.ps.layout, self.ps.world_size, 2 if self.ps.dtype == BF else 4, d0, inner,
                                        group_num_params=self.ps.groups)
        self.total = self.plan.info().total_numel
        self.shards = self.packed(W.make_params(self.ps))
        self.grads = [self.packed(g) for g in W.make_rank_grads(self.ps)]
        self.master = torch.empty(self.total, device="cuda") if with_master else None
        m = self.master if with_master else torch.empty(self.total, device="cuda")
        self.m, self.v = torch.empty(self.total, device="cuda"), torch.empty(self.total, device="cuda")
        ss.fsdp_init_master(self.plan, self.shards, m, self.m, self.v)
        self.norm = torch.empty(2, device="cuda")

    def packed(self, ts):
        buf = torch.empty(self.total, dtype=self.ps.dtype, device="cuda")
        self.ss.fsdp_pack(self.plan, [t.cuda() for t in ts], buf)
        return buf

    def state(self):
        return [t.clone() for t in (self.master, self.m, self.v, self.shards) if t is not None]

    def reduced(self):
        out = torch.empty(self.total, device="cuda")
        self.ss.fsdp_reduce_scatter_adamw(self.plan, self.grads, None, None, None, None, None, out)
        return out


@gpu
@pytest.mark.parametrize("by_group", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_reduce_scatter_norm(ss, kind, by_group):
    s = Sharded(ss, kind)
    G = len(s.ps.groups)
    red = torch.full((s.total,), 5.0, device="cuda")
    sq = torch.full((G if by_group else 1,), -1.0, dtype=torch.float64, device="cuda")
    ws = workspace(ss)
    for g in range(G) if by_group else [-1]:
        ss.fsdp_reduce_scatter_norm(s.plan, s.grads, red, sq[g if by_group else 0:], ws, group=g)
    want = s.reduced()
    assert torch.equal(red, want)
    for g in range(G) if by_group else [-1]:
        if by_group:
            grp = ss.fsdp_plan_group(s.plan, g)
            part = want[grp["base"]:grp["base"] + s.ps.world_size * grp["shard_numel"]]
        else:
            part = want
        w = float(part.double().square().sum())
        assert abs(float(sq[g if by_group else 0]) - w) <= 2 * NORM_RTOL * w


@gpu
@pytest.mark.parametrize("with_master", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_unclipped_is_the_plain_step(ss, kind, with_master):
    """With a factor of 1: state and shards bit for bit those of fsdp_reduce_scatter_adamw, over two steps."""
    a, b = Sharded(ss, kind, with_master), Sharded(ss, kind, with_master)
    red, sq = torch.empty(a.total, device="cuda"), torch.empty(1, dtype=torch.float64, device="cuda")
    ws = workspace(ss)
    for step in (1, 2):
        hp = ss.adamw_params(step=step)
        ss.fsdp_reduce_scatter_norm(a.plan, a.grads, red, sq, ws)
        ss.fsdp_clip_adamw(a.plan, red, sq, math.inf, a.master, a.m, a.v, a.shards, hp, a.norm)
        ss.fsdp_reduce_scatter_adamw(b.plan, b.grads, b.master, b.m, b.v, b.shards, hp)
    assert float(a.norm[1]) == 1.0
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)


@gpu
@pytest.mark.parametrize("kind", ["tiny", "flat_true_5_fp32"])
def test_unlimited_step_with_an_infinite_norm(ss, kind):
    """max_norm = +inf and a gradient whose square passes fp32: the plain step, bit for bit."""
    a, b = Sharded(ss, kind), Sharded(ss, kind)
    for s in (a, b):
        s.grads[0][5] = 3e38
    red, sq = torch.empty(a.total, device="cuda"), torch.empty(1, dtype=torch.float64, device="cuda")
    hp = ss.adamw_params()
    ss.fsdp_reduce_scatter_norm(a.plan, a.grads, red, sq, workspace(ss))
    ss.fsdp_clip_adamw(a.plan, red, sq, math.inf, a.master, a.m, a.v, a.shards, hp, a.norm)
    ss.fsdp_reduce_scatter_adamw(b.plan, b.grads, b.master, b.m, b.v, b.shards, hp)
    assert a.norm.tolist() == [math.inf, 1.0]
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)
    assert bool(a.master.isfinite().any())


@gpu
@pytest.mark.parametrize("by_group", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_clipped_step(ss, kind, by_group):
    """Against AdamW in 64 bits on the clipped mean; by group, the norm still spans all groups."""
    s = Sharded(ss, kind)
    G = len(s.ps.groups)
    red = torch.empty(s.total, device="cuda")
    sq = torch.empty(G if by_group else 1, dtype=torch.float64, device="cuda")
    ws = workspace(ss)
    want_norm = norm64([s.reduced()])
    max_norm = 0.3 * want_norm
    for step in (1, 2, 3):
        prev = [t.double().cpu().numpy() for t in (s.master, s.m, s.v)]
        hp = ss.adamw_params(step=step)
        for g in range(G) if by_group else [-1]:
            ss.fsdp_reduce_scatter_norm(s.plan, s.grads, red, sq[g if by_group else 0:], ws, group=g)
        for g in range(G) if by_group else [-1]:
            ss.fsdp_clip_adamw(s.plan, red, sq, max_norm, s.master, s.m, s.v, s.shards, hp, s.norm, group=g)
        n, c = (float(x) for x in s.norm)
        assert abs(n - want_norm) <= NORM_RTOL * want_norm
        c64 = max_norm / (want_norm + 1e-6)
        assert abs(c - c64) <= NORM_RTOL * c64
        # AdamW on the fp32 product with the factor the GPU reported
        grad = (red * c).double().cpu().numpy()
        th, m, v = prev
        m = 0.9 * m + 0.1 * grad
        v = 0.999 * v + 0.001 * grad * grad
        th = th * (1 - 1e-3 * 0.01)
        th = th - 1e-3 * (m / (1 - 0.9 ** step)) / (np.sqrt(v / (1 - 0.999 ** step)) + 1e-8)
        check_adamw_state(s.master.cpu().numpy(), s.m.cpu().numpy(), s.v.cpu().numpy(), th, m, v, prev[0], prev[1],
                          grad)
        assert torch.equal(s.shards, s.master.to(s.ps.dtype))


# Groups of more than 608 CTAs' work in either type (1.25 M bf16 elements), which take the factor from a launch of its
# own, with ranges that start and end inside a 16-byte vector.
def large_plan(dtype):
    return W.ParamSet([f"p{i}" for i in range(5)], [(1301, 1003), (7,), (1399, 1001), (5,), (3,)], [2, 2, 1], 3,
                      W.PER_PARAM_DIM0, dtype, seed=9, uniform=True)


@pytest.fixture(params=[BF, F32], ids=["bf16", "fp32"])
def large(request, monkeypatch):
    monkeypatch.setitem(globals(), "plan_of", lambda ss, kind: large_plan(request.param))


@gpu
@pytest.mark.parametrize("by_group", [False, True])
def test_large_reduce_scatter_norm(ss, large, by_group):
    test_reduce_scatter_norm(ss, "large", by_group)


@gpu
@pytest.mark.parametrize("with_master", [True, False])
def test_large_unclipped_is_the_plain_step(ss, large, with_master):
    test_unclipped_is_the_plain_step(ss, "large", with_master)


@gpu
@pytest.mark.parametrize("by_group", [False, True])
def test_large_clipped_step(ss, large, by_group):
    test_clipped_step(ss, "large", by_group)


@gpu
@pytest.mark.parametrize("with_master", [True, False])
def test_large_groups_are_the_whole_plan(ss, large, with_master):
    """Clipped by the same sums, the groups one by one and the plan at once give the same bits, with and without master,
    on one stream with nothing between the calls."""
    a, b = Sharded(ss, "large", with_master), Sharded(ss, "large", with_master)
    G = len(a.ps.groups)
    sq = torch.empty(G, dtype=torch.float64, device="cuda")
    ws = workspace(ss)
    red = torch.empty(a.total, device="cuda")
    for step in (1, 2):
        hp = ss.adamw_params(step=step)
        for g in range(G):
            ss.fsdp_reduce_scatter_norm(a.plan, a.grads, red, sq[g:], ws, group=g)
        for g in range(G):
            ss.fsdp_clip_adamw(a.plan, red, sq, 0.1, a.master, a.m, a.v, a.shards, hp, a.norm, group=g)
        ss.fsdp_clip_adamw(b.plan, red, sq, 0.1, b.master, b.m, b.v, b.shards, hp, b.norm)
    assert torch.equal(a.norm, b.norm) and float(a.norm[1]) < 1.0
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)


@gpu
def test_reduce_scatter_norm_past_32_bits(ss):
    """More than 2^31 elements, and more CTAs than partials: the mean of two equal ranks is either, bit for bit."""
    n = (1 << 31) + 8_000_003
    plan = ss.fsdp_plan_create(W.FLAT_ORIG_FALSE, 2, 2, [n], [1])
    total = plan.info().total_numel
    grad, block, sq = repeated(total, BF)
    red = torch.empty(total, device="cuda")
    out = torch.empty(1, dtype=torch.float64, device="cuda")
    ss.fsdp_reduce_scatter_norm(plan, [grad, grad], red, out, workspace(ss))
    assert abs(float(out[0]) - sq) <= 2 * HUGE_RTOL * sq
    wide = block.float()
    for a in range(0, total, 1 << 26):
        assert torch.equal(red[a:a + (1 << 26)], wide[:min(1 << 26, total - a)]), a
    plan.destroy()


@gpu
def test_norm_over_two_plans(ss):
    """The sums of two plans given together clip both by one norm."""
    a, b = Sharded(ss, "tiny"), Sharded(ss, "flat_false_7")
    sq = torch.empty(2, dtype=torch.float64, device="cuda")
    ws = workspace(ss)
    for k, s in enumerate((a, b)):
        s.red = torch.empty(s.total, device="cuda")
        ss.fsdp_reduce_scatter_norm(s.plan, s.grads, s.red, sq[k:], ws)
    want = norm64([a.red, b.red])
    for s in (a, b):
        ss.fsdp_clip_adamw(s.plan, s.red, sq, 0.5, s.master, s.m, s.v, s.shards, ss.adamw_params(), s.norm)
        assert abs(float(s.norm[0]) - want) <= NORM_RTOL * want
    assert torch.equal(a.norm, b.norm)


# ---------------------------------------------------------------------------
# refusals: all found on the host, before anything is launched
# ---------------------------------------------------------------------------

def status(ss, call):
    with pytest.raises(ss.ShardStateError) as e:
        call()
    return e.value.status


@gpu
def test_refusals(ss):
    ts, _ = tensors([100], [BF], [0])
    norm, ws = torch.empty(2, device="cuda"), workspace(ss)
    for bad in (-1.0, math.nan):
        assert status(ss, lambda: ss.ss_clip_grads(ts, bad, norm, ws)) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads(ts, 1.0, norm, ws[:1024])) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads(ts, 1.0, norm[:1], ws)) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads([ts[0].half()], 1.0, norm, ws)) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads([ts[0].cpu()], 1.0, norm, ws)) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads(ts, 1.0, norm.cpu(), ws)) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_grad_norm(ts, norm, ws.cpu())) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads([ts[0][::2]], 1.0, norm, ws)) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads(ts, 1.0, norm, ws, out=[])) == ss.SS_EINVAL
    assert status(ss, lambda: ss.ss_clip_grads(ts, 1.0, norm, ws, out=[ts[0].float()])) == ss.SS_EINVAL
    big = torch.empty(ss.SS_NORM_WORKSPACE_BYTES + 16, dtype=torch.uint8, device="cuda")
    assert status(ss, lambda: ss.ss_grad_norm(ts, norm, big[8:])) == ss.SS_EALIGN
    s = Sharded(ss, "tiny")
    launched = ss.ss_launch_count()  # of refused calls: none
    red, sq = torch.empty(s.total + 4, device="cuda"), torch.empty(1, dtype=torch.float64, device="cuda")
    rs = lambda **k: ss.fsdp_reduce_scatter_norm(**{**dict(plan=s.plan, rank_grads=s.grads, reduced_grad=red,
                                                           sq_out=sq, workspace=ws), **k})
    assert status(ss, lambda: rs(group=1)) == ss.SS_EINVAL
    assert status(ss, lambda: rs(reduced_grad=None)) == ss.SS_EINVAL
    assert status(ss, lambda: rs(reduced_grad=red[1:])) == ss.SS_EALIGN
    assert status(ss, lambda: rs(rank_grads=[s.grads[0], None])) == ss.SS_EINVAL
    assert status(ss, lambda: rs(workspace=ws[16:])) == ss.SS_EINVAL
    assert status(ss, lambda: rs(sq_out=sq.float())) == ss.SS_EINVAL
    ca = lambda **k: ss.fsdp_clip_adamw(**{**dict(
        plan=s.plan, reduced_grad=red, sq_sums=sq, max_norm=1.0, master=s.master, exp_avg=s.m, exp_avg_sq=s.v,
        param_shards=s.shards, hp=ss.adamw_params(), norm_out=norm), **k})
    assert status(ss, lambda: ca(max_norm=-1.0)) == ss.SS_EINVAL
    assert status(ss, lambda: ca(max_norm=math.nan)) == ss.SS_EINVAL
    assert status(ss, lambda: ca(hp=ss.adamw_params(step=0))) == ss.SS_EINVAL
    assert status(ss, lambda: ca(hp=ss.adamw_params(beta1=1.0))) == ss.SS_EINVAL
    assert status(ss, lambda: ca(exp_avg=None)) == ss.SS_EINVAL
    assert status(ss, lambda: ca(reduced_grad=red[1:])) == ss.SS_EALIGN
    assert status(ss, lambda: ca(group=7)) == ss.SS_EINVAL
    assert status(ss, lambda: ca(sq_sums=sq[:0])) == ss.SS_EINVAL
    assert ss.ss_launch_count() == launched


def test_refusals_on_the_host(ss):
    """What needs no device: bad counts, sizes, types and pointers through the C ABI."""
    import ctypes
    lib = ss.lib()
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    buf = ctypes.c_void_p(1 << 20)  # never touched
    ws, n = ctypes.c_void_p(1 << 30), ss.SS_NORM_WORKSPACE_BYTES

    def norm(count=1, numels=(8,), eb=(2,), ptrs=(1 << 20,), out=buf, workspace=ws, size=n):
        return lib.ss_grad_norm(count, (i64 * 4)(*numels), (i32 * 4)(*eb), (vp * 4)(*ptrs), out, workspace, size, None)

    assert norm(count=-1) == ss.SS_EINVAL
    assert norm(numels=(-1,)) == ss.SS_EINVAL
    assert norm(eb=(8,)) == ss.SS_EINVAL
    assert norm(ptrs=(0,)) == ss.SS_EINVAL
    assert norm(ptrs=((1 << 20) + 1,)) == ss.SS_EALIGN
    assert norm(eb=(4,), ptrs=((1 << 20) + 2,)) == ss.SS_EALIGN
    assert norm(numels=(2 ** 62,)) == ss.SS_EOVERFLOW
    assert norm(out=None) == ss.SS_EINVAL
    assert norm(workspace=None) == ss.SS_EINVAL
    assert norm(size=n - 1) == ss.SS_EINVAL
    assert lib.ss_grad_norm(1, None, None, None, buf, ws, n, None) == ss.SS_EINVAL
    plan = ss.fsdp_plan_create(0, 2, 2, [8], host_only=True)
    grads = (vp * 2)(1 << 20, 1 << 20)
    hp = ss.adamw_params()
    assert lib.fsdp_reduce_scatter_norm(plan, grads, buf, buf, ws, n, -1, None) == ss.SS_ENODEVICE
    assert lib.fsdp_clip_adamw(plan, buf, buf, 1, 1.0, None, buf, buf, buf, ctypes.byref(hp), buf, -1,
                               None) == ss.SS_ENODEVICE
    plan.destroy()
