"""The operators between a model's last hidden states and its clipped update, as cases to measure.

Three kinds of case:
  * "loss": linear cross entropy -- the LM head's product, the softmax cross entropy over the vocabulary and, for
    training, the gradients of hidden states and head weight, with no logits kept;
  * "clip": the global norm over a list of gradient tensors, and the clipped gradients;
  * "step": the sharded step with clipping -- reduce-scatter of N ranks' gradients with the sum of squares, then
    AdamW on the clipped mean.

`run` computes them in elementary torch operations where `own` is false, and through the package's entry points
where it is true.
"""
import math

import torch

own = False

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=10)
CLIP_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token scored against the 1.2B configuration's vocabulary: the read of the head's weight
        dict(name="loss_score_one_token", kind="loss", tokens=1, vocab=32000, hidden=2048, ignored=0, train=False),
        # a toy model's step: nothing but latency
        dict(name="loss_train_tiny", kind="loss", tokens=50, vocab=128, hidden=64, ignored=3, train=True),
        # a packed batch with its prompts masked out, an odd vocabulary and an odd hidden size
        dict(name="loss_train_ragged", kind="loss", tokens=1021, vocab=32003, hidden=1001, ignored=417, train=True),
        # one sequence of the 1.2B configuration
        dict(name="loss_train_2k", kind="loss", tokens=2048, vocab=32000, hidden=2048, ignored=0, train=True),
        # a whole micro-batch of it
        dict(name="loss_train_8k", kind="loss", tokens=8192, vocab=32000, hidden=2048, ignored=24, train=True),
        # evaluation at hidden 4096: per-token losses, no gradient
        dict(name="loss_score_4k", kind="loss", tokens=4096, vocab=32000, hidden=4096, ignored=1, train=False),
        # the tiny two-matrix MLP's five gradients
        dict(name="clip_tiny", kind="clip", model="tiny_mlp", count=5, mean=3328, fp32_every=0, max_norm=0.5),
        # 200 odd-sized tensors, a third of them fp32, at odd offsets of one buffer
        dict(name="clip_awkward", kind="clip", model="", count=200, mean=2500, fp32_every=3, max_norm=1.0),
        # every gradient of the 1.2B configuration
        dict(name="clip_model", kind="clip", model="llama_1b2", count=219, mean=6229670, fp32_every=0, max_norm=1.0),
        # the tiny MLP's sharded step, 2 ranks
        dict(name="step_tiny", kind="step", model="tiny_mlp", ranks=2, layout=1, count=5, mean=3328, fp32=False,
             max_norm=0.5),
        # 200 odd-sized parameters in one FlatParameter, 7 ranks
        dict(name="step_awkward", kind="step", model="", ranks=7, layout=0, count=200, mean=250001, fp32=False,
             max_norm=1.0),
        # the 1.2B configuration, 8 ranks, one group per block
        dict(name="step_model", kind="step", model="llama_1b2", ranks=8, layout=2, count=219, mean=6229670, fp32=False,
             max_norm=1.0),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["loss", "loss", "clip", "step"])
    if kind == "loss":
        tokens = _log_uniform(rng, 1, 8192)
        vocab = _log_uniform(rng, 128, 50000)
        hidden = _log_uniform(rng, 64, 3000) if rng.random() < 0.8 else rng.choice([3584, 4096])
        hidden = min(hidden, 8192 * 32000 * 2048 // (tokens * vocab))
        if rng.random() < 0.6:
            hidden = hidden // 8 * 8
        ignored = int(tokens * rng.choice([0.0, 0.0, 0.3, 0.7]) * rng.random())
        return dict(kind="loss", tokens=tokens, vocab=vocab, hidden=hidden, ignored=ignored,
                    train=rng.random() < 0.6)
    count = _log_uniform(rng, 1, 400)
    total = _log_uniform(rng, 2000, 1_200_000_000 if kind == "clip" else 600_000_000)
    mean = max(1, total // count)
    if kind == "clip":
        return dict(kind="clip", model="", count=count, mean=mean, fp32_every=rng.choice([0, 0, 1, 2, 5]),
                    max_norm=rng.choice([0.5, 1.0, 2.0]))
    return dict(kind="step", model="", ranks=rng.choice([1, 2, 3, 4, 5, 7, 8, 12]), layout=rng.choice([0, 1, 2]),
                count=count, mean=mean, fp32=rng.random() < 0.3, max_norm=rng.choice([0.5, 1.0, 2.0]))


def _shapes(case):
    """Parameter shapes of a clip or step case and the number of parameters in each group."""
    import workloads as W
    if case["model"] == "tiny_mlp":
        ps = W.tiny_mlp()
        return ps.shapes, ps.groups
    if case["model"] == "llama_1b2":
        ps = W.llama_1b2()
        return ps.shapes, ps.groups
    # lengths spread evenly over [1, 2 * mean), in a fixed scattered order, all of them odd sizes for the most part
    n, mean = case["count"], case["mean"]
    lens = [1 + ((2 * i + 1) * (mean - 1)) // n for i in range(n)]
    order = sorted(range(n), key=lambda i: (i * 7919 + 13) % 10007)
    return [(lens[i],) for i in order], [n]


def _numel(shape):
    return math.prod(shape)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(numel, std, dtype, gen):
    out = torch.empty(numel, dtype=dtype, device="cuda")
    piece = 1 << 28
    for a in range(0, numel, piece):
        b = min(numel, a + piece)
        out[a:b] = torch.randn(b - a, generator=gen, device="cuda") * std
    return out


def _views(flat, sizes):
    """Consecutive views of `flat`, one of each size."""
    out, at = [], 0
    for n in sizes:
        out.append(flat[at:at + n])
        at += n
    return out


def _loss_inputs(case, seed):
    """Hidden states of unit scale and a head of N(0, 0.02), the target's own logit raised by 0 to 12 (a model
    between its start and the end of its training); `ignored` targets are -100."""
    gen = torch.Generator("cuda").manual_seed(seed)
    T, V, D = case["tokens"], case["vocab"], case["hidden"]
    weight = _randn(V * D, 0.02, torch.bfloat16, gen).view(V, D)
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    rows = weight[targets].float()
    rise = torch.rand(T, 1, generator=gen, device="cuda") * 12.0
    hidden = torch.randn(T, D, generator=gen, device="cuda") + rise * rows / rows.square().sum(1, keepdim=True)
    away = torch.randperm(T, generator=gen, device="cuda")[:case["ignored"]]
    targets[away] = -100
    return hidden.to(torch.bfloat16), weight, targets


def _clip_inputs(case, seed):
    """Gradient tensors of N(0, 1e-2): bf16 and, where asked, every so many an fp32 one, cut one after another from
    one buffer per type (so at any element offset)."""
    gen = torch.Generator("cuda").manual_seed(seed)
    shapes, _ = _shapes(case)
    sizes = [_numel(s) for s in shapes]
    every = case["fp32_every"]
    is32 = [every > 0 and i % every == 0 for i in range(len(sizes))]
    n16 = sum(n for n, f in zip(sizes, is32) if not f)
    n32 = sum(n for n, f in zip(sizes, is32) if f)
    flat16 = _randn(n16, 1e-2, torch.bfloat16, gen)
    flat32 = _randn(n32, 1e-2, torch.float32, gen)
    return sizes, is32, flat16, flat32


def _step_inputs(case, seed):
    """Packed rank gradients (pads zero, as packing leaves them), fp32 state and shards of a plan."""
    import sharded_state_gb300 as ss
    gen = torch.Generator("cuda").manual_seed(seed)
    shapes, groups = _shapes(case)
    dtype = torch.float32 if case["fp32"] else torch.bfloat16
    d0 = [s[0] for s in shapes]
    inner = [_numel(s[1:]) for s in shapes]
    plan = ss.fsdp_plan_create(case["layout"], case["ranks"], 4 if case["fp32"] else 2, d0, inner,
                               group_num_params=groups)
    total = plan.info().total_numel
    sizes = [_numel(s) for s in shapes]

    def packed(std):
        buf = torch.empty(total, dtype=dtype, device="cuda")
        ss.fsdp_pack(plan, _views(_randn(sum(sizes), std, dtype, gen), sizes), buf)
        return buf

    shards = packed(0.02)
    grads = [packed(1e-2) for _ in range(case["ranks"])]
    master = shards.float()
    if not case["fp32"]:  # what training has moved the master by since the last rounding
        master += master * (torch.rand(total, generator=gen, device="cuda") - 0.5) * 2.0 ** -9
    exp_avg = torch.randn(total, generator=gen, device="cuda") * 1e-3
    exp_avg_sq = torch.rand(total, generator=gen, device="cuda") * 1e-5
    live = (shards != 0).float()  # pads hold zero state
    exp_avg *= live
    exp_avg_sq *= live
    return plan, grads, shards, master, exp_avg, exp_avg_sq


def prepare(case, seed):
    import sharded_state_gb300 as ss
    s = {"case": case}
    if case["kind"] == "loss":
        s["hidden"], s["weight"], s["targets"] = _loss_inputs(case, seed)
        T, V, D = case["tokens"], case["vocab"], case["hidden"]
        s["loss"] = torch.empty(1, device="cuda")
        s["token_loss"] = torch.empty(T, device="cuda")
        if case["train"]:
            s["d_hidden"] = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
            s["d_weight"] = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
        if hasattr(ss, "ss_linear_ce_workspace"):
            s["workspace"] = torch.empty(ss.ss_linear_ce_workspace(T, D, V, case["train"]), dtype=torch.uint8,
                                         device="cuda")
    elif case["kind"] == "clip":
        sizes, is32, flat16, flat32 = _clip_inputs(case, seed)
        out16, out32 = torch.empty_like(flat16), torch.empty_like(flat32)

        def tensors(a16, a32):
            v16 = iter(_views(a16, [n for n, f in zip(sizes, is32) if not f]))
            v32 = iter(_views(a32, [n for n, f in zip(sizes, is32) if f]))
            return [next(v32 if f else v16) for f in is32]

        s.update(flat16=flat16, flat32=flat32, out16=out16, out32=out32, grads=tensors(flat16, flat32),
                 out=tensors(out16, out32), norm=torch.empty(2, device="cuda"))
        if hasattr(ss, "GradClip"):
            s["workspace"] = torch.empty(ss.SS_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
            s["call"] = ss.GradClip(s["grads"], case["max_norm"], s["norm"], s["workspace"], out=s["out"])
    else:
        plan, grads, shards, master, exp_avg, exp_avg_sq = _step_inputs(case, seed)
        s.update(plan=plan, grads=grads, shards=shards, master=master, exp_avg=exp_avg, exp_avg_sq=exp_avg_sq,
                 grad_ptrs=ss.ptr_array(grads), reduced=torch.empty_like(master),
                 sq=torch.empty(1, dtype=torch.float64, device="cuda"), norm=torch.empty(2, device="cuda"),
                 hp=ss.adamw_params(**HYPER))
        if hasattr(ss, "SS_NORM_WORKSPACE_BYTES"):
            s["workspace"] = torch.empty(ss.SS_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"loss": _own_loss, "clip": _own_clip, "step": _own_step}[kind](s)
    return {"loss": _plain_loss, "clip": _plain_clip, "step": _plain_step}[kind](s)


def _own_loss(s):
    import sharded_state_gb300 as ss
    train = s["case"]["train"]
    ss.ss_linear_cross_entropy(s["hidden"], s["weight"], s["targets"], s["loss"], s["workspace"],
                               token_loss_out=s["token_loss"], d_hidden=s["d_hidden"] if train else None,
                               d_weight=s["d_weight"] if train else None)
    return _loss_outputs(s)


def _loss_outputs(s):
    out = {"loss": s["loss"], "token_loss": s["token_loss"]}
    if s["case"]["train"]:
        out.update(d_hidden=s["d_hidden"], d_weight=s["d_weight"])
    return out


def _own_clip(s):
    s["call"]()
    return {"out16": s["out16"], "out32": s["out32"], "norm": s["norm"]}


def _own_step(s):
    import sharded_state_gb300 as ss
    ss.fsdp_reduce_scatter_norm(s["plan"], s["grad_ptrs"], s["reduced"], s["sq"], s["workspace"])
    ss.fsdp_clip_adamw(s["plan"], s["reduced"], s["sq"], s["case"]["max_norm"], s["master"], s["exp_avg"],
                       s["exp_avg_sq"], s["shards"], s["hp"], s["norm"])
    return _step_outputs(s)


def _step_outputs(s):
    return {k: s[k] for k in ("reduced", "norm", "master", "exp_avg", "exp_avg_sq", "shards")}


def _plain_loss(s):
    hidden, weight, targets = s["hidden"].float(), s["weight"].float(), s["targets"]
    valid = targets != -100
    at = torch.where(valid, targets, 0).unsqueeze(1)
    p = hidden @ weight.t()
    top = p.amax(1, keepdim=True)
    target_logit = p.gather(1, at)
    p = p.sub_(top).exp_()
    total = p.sum(1, keepdim=True)
    token_loss = torch.where(valid, (top + total.log() - target_logit).squeeze(1), 0.0)
    count = valid.sum().clamp(min=1)
    s["token_loss"].copy_(token_loss)
    s["loss"].copy_(token_loss.sum() / count)
    if s["case"]["train"]:
        p = p.div_(total)
        p = p.scatter_add_(1, at, torch.full_like(target_logit, -1.0))
        p = p.mul_(valid.unsqueeze(1) / count)
        s["d_hidden"].copy_(p @ weight)
        s["d_weight"].copy_(p.t() @ hidden)
    return _loss_outputs(s)


def _plain_clip(s):
    x16, x32 = s["flat16"].float(), s["flat32"]
    norm = ((x16 * x16).sum() + (x32 * x32).sum()).sqrt()
    factor = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    s["out16"].copy_(x16 * factor)
    s["out32"].copy_(x32 * factor)
    s["norm"].copy_(torch.stack([norm, factor]))
    return {"out16": s["out16"], "out32": s["out32"], "norm": s["norm"]}


def _plain_step(s):
    h = HYPER
    g = torch.zeros_like(s["master"])
    for x in s["grads"]:
        g += x
    g = g.div_(len(s["grads"]))
    norm = (g * g).sum().sqrt()
    factor = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    s["reduced"].copy_(g)
    s["norm"].copy_(torch.stack([norm, factor]))
    g = g.mul_(factor)
    m, v, w = s["exp_avg"], s["exp_avg_sq"], s["master"]
    m.mul_(h["beta1"]).add_(g, alpha=1 - h["beta1"])
    v.mul_(h["beta2"]).addcmul_(g, g, value=1 - h["beta2"])
    c1, c2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    w.mul_(1 - h["lr"] * h["weight_decay"])
    w.sub_((h["lr"] / c1) * m / (v.sqrt() / math.sqrt(c2) + h["eps"]))
    s["shards"].copy_(w)
    return _step_outputs(s)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    return {"loss": _exact_loss, "clip": _exact_clip, "step": _exact_step}[case["kind"]](case, seed)


def _exact_loss(case, seed):
    hidden, weight, targets = _loss_inputs(case, seed)
    h, w = hidden.double(), weight.double()
    keep = torch.nonzero(targets >= 0).squeeze(1)
    n = max(1, keep.numel())
    hk, yk = h[keep], targets[keep]
    logp = torch.log_softmax(hk @ w.t(), dim=1)
    nll = -logp[torch.arange(keep.numel(), device="cuda"), yk]
    token_loss = torch.zeros(case["tokens"], dtype=torch.float64, device="cuda")
    token_loss[keep] = nll
    out = {"loss": (nll.sum() / n).reshape(1), "token_loss": token_loss}
    if case["train"]:
        d = logp.exp_()
        d[torch.arange(keep.numel(), device="cuda"), yk] -= 1.0
        d /= n
        dh = torch.zeros_like(h)
        dh[keep] = d @ w
        out.update(d_hidden=dh, d_weight=d.t() @ hk)
    return out


def _exact_clip(case, seed):
    _, _, flat16, flat32 = _clip_inputs(case, seed)
    a, b = flat16.double(), flat32.double()
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(a), torch.linalg.vector_norm(b)]))
    factor = torch.clamp(case["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return {"out16": a.mul_(factor), "out32": b.mul_(factor), "norm": torch.stack([norm, factor])}


def _exact_step(case, seed):
    h = HYPER
    _, grads, _, master, exp_avg, exp_avg_sq = _step_inputs(case, seed)
    g = torch.zeros(master.numel(), dtype=torch.float64, device="cuda")
    for x in grads:
        g += x
    del grads
    g /= case["ranks"]
    norm = torch.linalg.vector_norm(g)
    factor = torch.clamp(case["max_norm"] / (norm + CLIP_EPS), max=1.0)
    out = {"reduced": g.clone(), "norm": torch.stack([norm, factor])}
    g *= factor
    m = exp_avg.double() * h["beta1"] + g * (1 - h["beta1"])
    v = exp_avg_sq.double() * h["beta2"] + g.square_() * (1 - h["beta2"])
    w = master.double() * (1 - h["lr"] * h["weight_decay"])
    m_hat = m / (1 - h["beta1"] ** h["step"])
    w -= h["lr"] * m_hat / ((v / (1 - h["beta2"] ** h["step"])).sqrt_() + h["eps"])
    out.update(master=w, exp_avg=m, exp_avg_sq=v, shards=w)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["kind"] == "loss":
        T, V, D, live = case["tokens"], case["vocab"], case["hidden"], case["tokens"] - case["ignored"]
        grad = 2.0 * (T * D + V * D) if case["train"] else 0.0
        return {"bytes": 2.0 * (live * D + V * D) + 8.0 * T + 4.0 * T + 4.0 + grad,
                "flops": (6.0 if case["train"] else 2.0) * live * V * D}
    shapes, _ = _shapes(case)
    n = sum(_numel(s) for s in shapes)
    if case["kind"] == "clip":
        every = case["fp32_every"]
        wide = sum(_numel(s) for i, s in enumerate(shapes) if every > 0 and i % every == 0)
        return {"bytes": 4.0 * (n - wide) + 8.0 * wide, "flops": 3.0 * n}
    e = 4 if case["fp32"] else 2
    return {"bytes": float(n) * (case["ranks"] * e + 12 + 4 + 12 + e), "flops": float(n) * (case["ranks"] + 20)}
