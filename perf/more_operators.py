"""The operators of a trained layer's residual stream and of its products in few bits, as cases to measure.

Four kinds of case:
  * "dropout": dropout whose mask comes from a counter-based generator and is never stored;
  * "norm": the root-mean-square norm of a residual stream -- dropout of the branch, the residual's addition, the
    norm -- and its backward pass, as a training step makes them;
  * "quant": microscaled quantisation (4-bit or 8-bit elements, a power of two for each 32) and back;
  * "linear": a product of quantised activations with a quantised weight: for a user's tokens with the weight kept
    in 4 or 8 bits, behind a norm that writes 8 bits itself, or as a training step's three products.

`run` computes them in elementary torch operations where `own` is false, and through the package's entry points
where it is true.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
FORMATS = {"mxfp4": 0, "mxfp8": 1}
# exponent of the largest element, lowest exponent, fraction bits, largest element
ELEMENT = {"mxfp4": (2, 0, 1, 6.0), "mxfp8": (8, -6, 3, 448.0)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 32  # elements that share a scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the hidden layer of an MLP block at FFN 11008, a micro-batch of 8192 tokens
        dict(name="dropout_ffn", kind="dropout", rows=8192, cols=11008, fp32=False, p=0.1),
        # odd sizes in fp32
        dict(name="dropout_ragged", kind="dropout", rows=1021, cols=1001, fp32=True, p=0.25),
        # a toy model's step: nothing but latency
        dict(name="norm_train_tiny", kind="norm", rows=50, cols=64, fp32=False, p=0.1),
        # a packed batch at an odd hidden size
        dict(name="norm_train_ragged", kind="norm", rows=1021, cols=1001, fp32=False, p=0.1),
        # a micro-batch at hidden 4096, trained without dropout
        dict(name="norm_train_16k", kind="norm", rows=16384, cols=4096, fp32=False, p=0.0),
        # the 1.2B configuration's head: what a gather of quantised weights sends, and what comes out of it
        dict(name="quant_head", kind="quant", rows=32000, cols=2048, fp32=False, format="mxfp4"),
        # an odd fp32 master weight in 8 bits
        dict(name="quant_ragged", kind="quant", rows=2043, cols=1001, fp32=True, format="mxfp8"),
        # one token through an up projection kept in 4 bits: the read of the weight
        dict(name="linear_token", kind="linear", tokens=1, inner=4096, outer=11008, format="mxfp4", norm=False,
             train=False),
        # odd sizes throughout
        dict(name="linear_ragged", kind="linear", tokens=1021, inner=1001, outer=777, format="mxfp4", norm=False,
             train=False),
        # residual, norm and up projection of one sequence of the 1.2B configuration, in 8 bits
        dict(name="linear_norm_2k", kind="linear", tokens=2048, inner=2048, outer=5632, format="mxfp8", norm=True,
             train=False),
        # a micro-batch through the up projection at hidden 4096, in 4 bits
        dict(name="linear_8k", kind="linear", tokens=8192, inner=4096, outer=11008, format="mxfp4", norm=False,
             train=False),
        # the 1.2B configuration's up projection trained in 4 bits: forward, both gradients
        dict(name="linear_train_8k", kind="linear", tokens=8192, inner=2048, outer=5632, format="mxfp4", norm=False,
             train=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["dropout", "norm", "norm", "quant", "linear", "linear", "linear"])
    if kind == "linear":
        tokens = _log_uniform(rng, 1, 8192)
        inner = _log_uniform(rng, 64, 4096)
        outer = _log_uniform(rng, 64, 11008)
        if rng.random() < 0.6:
            inner, outer = inner // 32 * 32, outer // 8 * 8
        format = rng.choice(["mxfp4", "mxfp4", "mxfp8"])
        mode = rng.random()
        if mode < 0.4:
            tokens = min(tokens, 8192 * 4096 * 11008 // (3 * inner * outer))
        return dict(kind="linear", tokens=tokens, inner=inner, outer=outer, format=format,
                    norm=mode >= 0.4 and format == "mxfp8" and rng.random() < 0.6, train=mode < 0.4)
    rows, cols = _log_uniform(rng, 1, 32000), _log_uniform(rng, 17, 11008)
    rows = min(rows, 16384 * 4096 // cols)
    if rng.random() < 0.6:
        cols = max(8, cols // 8 * 8)
    fp32 = rng.random() < 0.3
    if kind == "quant":
        return dict(kind="quant", rows=rows, cols=cols, fp32=fp32, format=rng.choice(["mxfp4", "mxfp8"]))
    return dict(kind=kind, rows=rows, cols=cols, fp32=fp32,
                p=rng.choice([0.05, 0.1, 0.5]) if kind == "dropout" or rng.random() < 0.6 else 0.0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _dtype(case):
    return torch.float32 if case.get("fp32") else torch.bfloat16


def _randn(rows, cols, std, dtype, gen):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(dtype)


def _rng(gen):
    """{seed, offset} of the counter-based generator, as a program keeps it on the device."""
    return torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")


def _inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, kind = _dtype(case), case["kind"]
    if kind == "dropout":
        return {"x": _randn(case["rows"], case["cols"], 1.0, dtype, gen), "rng": _rng(gen)}
    if kind == "norm":
        rows, cols = case["rows"], case["cols"]
        s = {name: _randn(rows, cols, std, dtype, gen)
             for name, std in (("x", 1.0), ("residual", 2.0), ("d_out", 1e-2), ("d_sum", 1e-2))}
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
        s["rng"] = _rng(gen)
        return s
    if kind == "quant":
        return {"x": _randn(case["rows"], case["cols"], 0.02, dtype, gen)}
    T, K, N = case["tokens"], case["inner"], case["outer"]
    # activations with channels of unlike scale, as a trained model's have
    channel = torch.exp2(torch.randn(K, generator=gen, device="cuda"))
    s = {"x": (torch.randn(T, K, generator=gen, device="cuda") * channel).to(dtype),
         "weight": _randn(N, K, 0.02, dtype, gen)}
    if case["norm"]:
        s["residual"] = _randn(T, K, 2.0, dtype, gen)
        s["norm_weight"] = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(dtype)
    if case["train"]:
        s["d_out"] = _randn(T, N, 1e-3, dtype, gen)
        s["rng"] = _rng(gen)
    return s


def _buffers(rows, cols, format):
    """Data (rows of whole 128 elements) and scales (512 bytes for each 128 x 128 elements) of a quantised matrix."""
    wide = -(-cols // 128)
    data = torch.empty(rows, wide * (64 if format == "mxfp4" else 128), dtype=torch.uint8, device="cuda")
    return data, torch.empty(-(-rows // 128) * wide * 512, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    kind, dtype = case["kind"], _dtype(case)
    if kind == "dropout":
        s["out"] = torch.empty_like(s["x"])
    elif kind == "norm":
        for name in ("sum", "out", "d_h") + (("d_x",) if case["p"] > 0 else ()):
            s[name] = torch.empty_like(s["x"])
        s["rstd"] = torch.empty(case["rows"], device="cuda")
        s["d_weight"] = torch.empty_like(s["weight"])
    elif kind == "quant":
        s["data"], s["scales"] = _buffers(case["rows"], case["cols"], case["format"])
        s["out"] = torch.empty_like(s["x"])
    else:
        T, K, N, format = case["tokens"], case["inner"], case["outer"], case["format"]
        s["x_q"] = _buffers(T, K, format)
        s["out"] = torch.empty(T, N, dtype=dtype, device="cuda")
        if case["train"]:
            s["w_q"] = _buffers(N, K, format)
            for name, rows, cols in (("x_t", K, T), ("w_t", K, N), ("d_q", T, N), ("d_t", N, T)):
                s[name] = _buffers(rows, cols, format)
            s["d_x"], s["d_w"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
        else:  # the weight is kept quantised
            s["w_q"] = _packed(s.pop("weight"), format)
        if case["norm"]:
            s["sum"] = torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------------------
# one pass through the package
# ---------------------------------------------------------------------------

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"dropout": _own_dropout, "norm": _own_norm, "quant": _own_quant, "linear": _own_linear}[kind](s)
    return {"dropout": _plain_dropout, "norm": _plain_norm, "quant": _plain_quant, "linear": _plain_linear}[kind](s)


def _own_dropout(s):
    import sharded_state_gb300 as ss
    ss.ss_dropout(s["x"], s["out"], s["case"]["p"], s["rng"])
    return s["out"]


def _own_norm(s):
    import sharded_state_gb300 as ss
    case = s["case"]
    if "workspace" not in s:  # kept from step to step
        n = ss.ss_rms_norm_workspace(case["rows"], case["cols"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    ss.ss_rms_norm(s["x"], s["weight"], EPS, out=s["out"], residual=s["residual"], sum_out=s["sum"],
                   rstd_out=s["rstd"], dropout=case["p"], rng=s["rng"])
    ss.ss_rms_norm_backward(s["d_out"], s["sum"], s["weight"], s["rstd"], s["d_h"], s["workspace"], d_sum=s["d_sum"],
                            d_x=s.get("d_x"), d_weight=s["d_weight"], dropout=case["p"], rng=s["rng"])
    return _norm_outputs(s)


def _norm_outputs(s):
    return {k: s[k] for k in ("out", "sum", "rstd", "d_h", "d_x", "d_weight") if k in s}


def _own_quant(s):
    import sharded_state_gb300 as ss
    format = FORMATS[s["case"]["format"]]
    ss.ss_mx_quantize(s["x"], format, s["data"], s["scales"])
    ss.ss_mx_dequantize(s["data"], s["scales"], format, s["out"])
    return s["out"]


def _own_linear(s):
    import sharded_state_gb300 as ss
    case = s["case"]
    T, K, N, format = case["tokens"], case["inner"], case["outer"], FORMATS[case["format"]]
    if case["train"]:
        ss.ss_mx_quantize(s["x"], format, *s["x_q"], *s["x_t"])
        ss.ss_mx_quantize(s["weight"], format, *s["w_q"], *s["w_t"])
        ss.ss_mx_matmul(*s["x_q"], *s["w_q"], K, format, s["out"])
        ss.ss_mx_quantize(s["d_out"], format, *s["d_q"], *s["d_t"], rng=s["rng"])
        ss.ss_mx_matmul(*s["d_q"], *s["w_t"], N, format, s["d_x"])
        ss.ss_mx_matmul(*s["d_t"], *s["x_t"], T, format, s["d_w"])
        return _linear_outputs(s)
    if case["norm"]:
        ss.ss_rms_norm(s["x"], s["norm_weight"], EPS, residual=s["residual"], sum_out=s["sum"], mx_data=s["x_q"][0],
                       mx_scales=s["x_q"][1])
    else:
        ss.ss_mx_quantize(s["x"], format, *s["x_q"])
    ss.ss_mx_matmul(*s["x_q"], *s["w_q"], K, format, s["out"])
    return _linear_outputs(s)


def _linear_outputs(s):
    return {k: s[k] for k in ("out", "sum", "d_x", "d_w") if k in s}


# ---------------------------------------------------------------------------
# the same in elementary operations
# ---------------------------------------------------------------------------

def _bits(rng, rows, cols):
    """16 random bits for each element of a matrix: Philox4x32-10 (Salmon et al., 2011) of key `seed` and counter
    {column / 8, row, offset}; its 128 bits are those of 8 columns, the lowest first."""
    low = 0xFFFFFFFF
    k0, k1 = rng[0] & low, rng[0] >> 32 & low
    groups = -(-cols // 8)
    a = torch.arange(groups, device="cuda").expand(rows, groups)
    b = torch.arange(rows, device="cuda")[:, None].expand(rows, groups)
    c, d = (rng[1] & low).expand(rows, groups), (rng[1] >> 32 & low).expand(rows, groups)
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57  # the low 64 bits, whatever their sign
        a, b, c, d = (y >> 32 & low) ^ b ^ k0, y & low, (x >> 32 & low) ^ d ^ k1, x & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack([a, b, c, d], 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).reshape(rows, 8 * groups)[:, :cols]


def _dropped(x, p, rng):
    """x in fp32 with its dropout, p in steps of 2^-16."""
    if p == 0:
        return x
    drop = round(p * 65536)
    keep = _bits(rng, *x.shape) >= drop
    return torch.where(keep, x * (65536 / (65536 - drop)), 0.0)


def _plain_dropout(s):
    s["out"].copy_(_dropped(s["x"].float(), s["case"]["p"], s["rng"]))
    return s["out"]


def _plain_norm(s):
    p, rng = s["case"]["p"], s["rng"]
    s["sum"].copy_(_dropped(s["x"].float(), p, rng) + s["residual"].float())
    h, w = s["sum"].float(), s["weight"].float()
    rstd = 1 / ((h * h).mean(1, keepdim=True) + EPS).sqrt()
    s["rstd"].copy_(rstd[:, 0])
    normed = h * rstd
    s["out"].copy_(normed * w)
    dy = s["d_out"].float()
    s["d_weight"].copy_((dy * normed).sum(0))
    g = dy * w
    d_h = rstd * (g - normed * (g * normed).mean(1, keepdim=True)) + s["d_sum"].float()
    s["d_h"].copy_(d_h)
    if p > 0:
        s["d_x"].copy_(_dropped(d_h, p, rng))
    return _norm_outputs(s)


def _codes(x, format, bits=None):
    """Elements (in units of their scale) and exponents of the scales of a matrix whose rows are cut in blocks of 32:
    the block's largest element gets the format's largest exponent.  Rounded to the nearest, ties to even, or up where
    the part cut off and the random bits / 2^16 make one.  Blocks that hold an infinity or a NaN are NaN."""
    top, lowest, fraction, most = ELEMENT[format]
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    largest = x.abs().amax(2, keepdim=True)
    bad = ~(largest < math.inf)
    x, largest = torch.where(bad, 0.0, x), torch.where(bad, 0.0, largest)
    scale = torch.where(largest > 0, torch.frexp(largest)[1] - 1 - top, -127).clamp(min=-127)
    v = torch.ldexp(x, -scale)
    size = v.abs()
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(size)[1] - 1).clamp(min=lowest) - fraction)
    step = torch.where(size > 0, step, 1.0)
    if bits is None:
        size = torch.round(size / step) * step
    else:
        bits = torch.nn.functional.pad(bits, (0, -cols % BLOCK)).view_as(x)
        size = torch.floor(size / step + bits * 2.0 ** -16) * step
    v = torch.copysign(size.clamp(max=most), v)
    return v, scale, bad


def _quantised(x, format, bits=None):
    """The values that the quantised matrix stands for."""
    v, scale, bad = _codes(x, format, bits)
    v = torch.where(bad, math.nan, torch.ldexp(v, scale))
    return v.reshape(x.shape[0], -1)[:, :x.shape[1]]


def _packed(x, format):
    """A quantised matrix as the package lays it out."""
    v, scale, bad = _codes(x, format)
    rows, cols = x.shape
    v = v.reshape(rows, -1)
    v = torch.nn.functional.pad(v, (0, -v.shape[1] % 128))
    if format == "mxfp4":
        code = torch.bucketize(v.abs(), torch.tensor(E2M1, device="cuda")) | torch.signbit(v).long() << 3
        data = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
    else:
        data = v.to(torch.float8_e4m3fn).view(torch.uint8)
    byte = torch.where(bad, 255, scale + 127)[:, :, 0]
    byte = torch.nn.functional.pad(byte, (0, -byte.shape[1] % 4, 0, -rows % 128)).to(torch.uint8)
    # tiles of 128 rows and 4 scales: row 32 i + j at 16 j + 4 i
    tiles = byte.view(byte.shape[0] // 128, 4, 32, byte.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return data.contiguous(), tiles.reshape(-1).contiguous()


def _unpacked(q, rows, cols, format):
    data, scales = q
    if format == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        v = torch.stack([table[(data & 15).long()], table[(data >> 4).long()]], 2)
    else:
        v = data.view(torch.float8_e4m3fn).float()
    wide = -(-cols // 128)
    byte = scales.view(-1, wide, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * wide)[:rows].int()
    factor = torch.where(byte == 255, math.nan, torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte - 127))
    return (v.view(rows, -1, BLOCK) * factor[:, :, None]).view(rows, -1)[:, :cols]


def _plain_quant(s):
    s["out"].copy_(_quantised(s["x"], s["case"]["format"]))
    return s["out"]


def _plain_linear(s):
    case = s["case"]
    T, K, N, format = case["tokens"], case["inner"], case["outer"], case["format"]
    if case["train"]:
        x, w, dy = s["x"], s["weight"], s["d_out"]
        bits = _bits(s["rng"], T, N)
        s["out"].copy_(_quantised(x, format) @ _quantised(w, format).t())
        s["d_x"].copy_(_quantised(dy, format, bits) @ _quantised(w.t(), format).t())
        s["d_w"].copy_(_quantised(dy.t(), format, bits.t()) @ _quantised(x.t(), format).t())
        return _linear_outputs(s)
    x = s["x"]
    if case["norm"]:
        s["sum"].copy_(x.float() + s["residual"].float())
        h = s["sum"].float()
        x = h * (1 / ((h * h).mean(1, keepdim=True) + EPS).sqrt()) * s["norm_weight"].float()
    s["out"].copy_(_quantised(x, format) @ _unpacked(s["w_q"], N, K, format).t())
    return _linear_outputs(s)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    return {"dropout": _exact_dropout, "norm": _exact_norm, "quant": _exact_quant,
            "linear": _exact_linear}[case["kind"]](case, s)


def _exact_bits(rng, rows, cols):
    seed, offset = (int(v) for v in rng.cpu())
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    groups = -(-cols // 8)
    x = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (rows, groups)).copy(),
         np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, groups)).copy(),
         np.full((rows, groups), offset & 0xFFFFFFFF, np.uint64), np.full((rows, groups), offset >> 32, np.uint64)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        k = [np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)]
        p, q = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(q >> half) ^ x[1] ^ k[0], q & low, (p >> half) ^ x[3] ^ k[1], p & low]
    out = np.empty((rows, groups, 8), np.int32)
    for i in range(4):
        out[:, :, 2 * i] = (x[i] & np.uint64(0xFFFF)).astype(np.int32)
        out[:, :, 2 * i + 1] = (x[i] >> np.uint64(16)).astype(np.int32)
    return torch.from_numpy(out.reshape(rows, 8 * groups)[:, :cols]).cuda()


def _exact_dropped(x, p, rng):
    drop = round(p * 65536)
    if not drop:
        return x
    return x * (_exact_bits(rng, *x.shape) >= drop) / (1 - drop / 65536)


def _exact_dropout(case, s):
    return _exact_dropped(s["x"].double(), case["p"], s["rng"])


def _exact_sum(x, residual, dtype):
    """The residual stream, which is stored in its type."""
    return (x + residual.double()).to(dtype).double()


def _exact_norm(case, s):
    rows, cols = case["rows"], case["cols"]
    h = _exact_sum(_exact_dropped(s["x"].double(), case["p"], s["rng"]), s["residual"], _dtype(case))
    w, dy = s["weight"].double(), s["d_out"].double()
    rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / cols + EPS)
    out = {"sum": h, "out": h / rms[:, None] * w, "rstd": 1 / rms}
    along = torch.einsum("rc,rc->r", dy * w, h)
    out["d_h"] = dy * w / rms[:, None] - h * (along / (cols * rms ** 3))[:, None] + s["d_sum"].double()
    out["d_weight"] = torch.einsum("rc,r->c", dy * h, 1 / rms)
    if case["p"] > 0:
        out["d_x"] = _exact_dropped(out["d_h"], case["p"], s["rng"])
    return out


def _exact_quantised(x, format, bits=None):
    """Every element of a block goes to one of the two values of the format's list that enclose it."""
    if format == "mxfp4":
        table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    else:
        table = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    full = torch.zeros(rows, blocks * BLOCK, dtype=torch.float64, device="cuda")
    full[:, :cols] = x
    full = full.view(rows, blocks, BLOCK)
    largest = full.abs().amax(2, keepdim=True)
    exponent = (largest.view(torch.int64) >> 52) - 1023  # of a normal fp64 number; 0 gives the lowest
    scale = torch.exp2((exponent - (2 if format == "mxfp4" else 8)).clamp(min=-127).double())
    v = (full / scale).abs()
    at = (torch.searchsorted(table, v, right=True) - 1).clamp(max=table.numel() - 2)
    below, above = table[at], table[at + 1]
    part = (v - below) / (above - below)
    if bits is None:
        up = (part > 0.5) | ((part == 0.5) & (at % 2 == 1))
    else:
        u = torch.zeros(rows, blocks * BLOCK, dtype=torch.float64, device="cuda")
        u[:, :cols] = bits / 65536.0
        up = part + u.view_as(v) >= 1
    v = torch.where(up, above, below)
    return (torch.sign(full) * v * scale).view(rows, -1)[:, :cols]


def _exact_quant(case, s):
    return _exact_quantised(s["x"].double(), case["format"])


def _exact_linear(case, s):
    format, x, w = case["format"], s["x"].double(), s["weight"].double()
    out = {}
    if case["norm"]:
        h = _exact_sum(x, s["residual"], _dtype(case))
        out["sum"] = h
        x = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["norm_weight"].double()
    out["out"] = _exact_quantised(x, format) @ _exact_quantised(w, format).t()
    if case["train"]:
        dy = s["d_out"].double()
        bits = _exact_bits(s["rng"], *dy.shape)
        out["d_x"] = _exact_quantised(dy, format, bits) @ _exact_quantised(w.t(), format).t()
        out["d_w"] = _exact_quantised(dy.t(), format, bits.t()) @ _exact_quantised(x.t(), format).t()
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _held(rows, cols, format):
    """Bytes of a quantised matrix."""
    return rows * cols * (0.5 if format == "mxfp4" else 1.0) + rows * -(-cols // BLOCK)


def work(case):
    if case["kind"] == "linear":
        T, K, N, format = case["tokens"], case["inner"], case["outer"], case["format"]
        if case["train"]:  # x, weight and d_out read, out and two gradients written
            return {"bytes": 2.0 * 2 * (T * K + N * K + T * N), "flops": 6.0 * T * N * K}
        extra = 2.0 * (2 * T * K + K) if case["norm"] else 0.0
        return {"bytes": 2.0 * T * K + extra + _held(N, K, format) + 2.0 * T * N, "flops": 2.0 * T * N * K}
    n, e = case["rows"] * case["cols"], 4 if case["fp32"] else 2
    if case["kind"] == "dropout":
        return {"bytes": 2.0 * n * e, "flops": 1.0 * n}
    if case["kind"] == "quant":  # out to the quantised form and back
        return {"bytes": 2.0 * n * e + 2 * _held(case["rows"], case["cols"], case["format"]), "flops": 4.0 * n}
    # forward: x and residual read, sum and out written; backward: d_out, d_sum and sum read, d_h (and d_x) written
    tensors = 4 + 4 + (1 if case["p"] > 0 else 0)
    return {"bytes": float(tensors * n * e + 4 * case["cols"] * e + 8 * case["rows"]), "flops": 20.0 * n}
