"""Plain 64-bit forms of dropout and microscaled floats, for the tests (numpy and torch, any device)."""
import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [(m / 8.0 if e == 0 else 1.0 + m / 8.0) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127]


def philox(counter, key):
    """Philox4x32-10 on Python integers: four words out of four words and two."""
    x, k = list(counter), list(key)
    for _ in range(10):
        p, q = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
        x = [(q >> 32) ^ x[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ x[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def bits16(seed, offset, rows, cols, row0=0, col0=0):
    """The 16 bits of each element from (row0, col0) on, int32 [rows, cols]; col0 a multiple of 8."""
    seed, offset = seed & (1 << 64) - 1, offset & (1 << 64) - 1
    groups = -(-cols // 8)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [np.broadcast_to(np.arange(col0 // 8, col0 // 8 + groups, dtype=np.uint64), (rows, groups)),
         np.broadcast_to(np.arange(row0, row0 + rows, dtype=np.uint64)[:, None], (rows, groups)),
         np.full((rows, groups), offset & 0xFFFFFFFF, np.uint64), np.full((rows, groups), offset >> 32, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        kk = [np.uint64((k[0] + r * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((k[1] + r * 0xBB67AE85) & 0xFFFFFFFF)]
        p, q = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(q >> half) ^ x[1] ^ kk[0], q & low, (p >> half) ^ x[3] ^ kk[1], p & low]
    out = np.empty((rows, groups, 8), np.int32)
    for i in range(4):
        out[:, :, 2 * i] = (x[i] & np.uint64(0xFFFF)).astype(np.int32)
        out[:, :, 2 * i + 1] = (x[i] >> np.uint64(16)).astype(np.int32)
    return torch.from_numpy(out.reshape(rows, groups * 8)[:, :cols].copy())


def keep_mask(rng, rows, cols, p, **at):
    seed, offset = (int(v) for v in rng.cpu())
    return bits16(seed, offset, rows, cols, **at) >= round(p * 65536)


def table(format):
    return torch.tensor(E2M1 if format == 0 else E4M3, dtype=torch.float64)


def quantise(x, format, bits=None):
    """(codes of the magnitudes, sign bits, stored scales) of x's rows, and the values they stand for: every element
    of a block of 32 goes to one of the two listed magnitudes around it."""
    x = x.detach().double().cpu()
    rows, cols = x.shape
    blocks = -(-cols // 32)
    full = torch.zeros(rows, blocks * 32, dtype=torch.float64)
    full[:, :cols] = x
    full = full.view(rows, blocks, 32)
    bad = ~torch.isfinite(full).all(2, keepdim=True)
    full = torch.where(bad, 0.0, full)
    top = full.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(torch.where(top > 0, top, 1.0))), -1000.0)
    # log2 may round up to a whole number just below a power of two
    e = torch.where((top > 0) & (torch.exp2(e) > top), e - 1, e)
    scale = (e - (2 if format == 0 else 8)).clamp(min=-127.0)
    v = full.abs() / torch.exp2(scale)
    t = table(format)
    at = (torch.searchsorted(t, v.contiguous(), right=True) - 1).clamp(max=len(t) - 2)
    below, above = t[at], t[at + 1]
    part = (v - below) / (above - below)
    if bits is None:
        up = (part > 0.5) | ((part == 0.5) & (at % 2 == 1))
    else:
        u = torch.zeros(rows, blocks * 32, dtype=torch.float64)
        u[:, :cols] = bits.double().cpu() / 65536
        up = part + u.view_as(v) >= 1
    code = at + up
    sign = torch.signbit(full)
    byte = torch.where(bad, 255.0, scale + 127).to(torch.int64)[:, :, 0]
    value = torch.where(sign, -t[code], t[code]) * torch.exp2(scale)
    value = torch.where(bad, float("nan"), value).view(rows, -1)[:, :cols]
    return code.view(rows, -1)[:, :cols], sign.view(rows, -1)[:, :cols], byte, value


def unpack(data, scales, rows, cols, format):
    """(codes of the magnitudes, sign bits, stored scales) as the two buffers hold them, the columns behind the last
    (to a multiple of 128) included."""
    wide = -(-cols // 128)
    data = data.cpu()[:rows * wide * (64 if format == 0 else 128)].view(rows, -1).to(torch.int64)
    if format == 0:
        c = torch.stack([data & 15, data >> 4], 2).view(rows, -1)
        code, sign = c & 7, c >> 3
    else:
        code, sign = data & 127, data >> 7
    flat = scales.cpu().to(torch.int64)
    r, b = torch.arange(rows)[:, None], torch.arange(4 * wide)[None, :]
    at = ((r // 128) * wide + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    return code, sign.bool(), flat[at]


def values(data, scales, rows, cols, format):
    """What the two buffers stand for, fp64 on the CPU."""
    code, sign, byte = unpack(data, scales, rows, cols, format)
    t = table(format)
    v = torch.where(sign, -t[code.clamp(max=len(t) - 1)], t[code.clamp(max=len(t) - 1)])
    factor = torch.where(byte == 255, float("nan"), torch.exp2(byte.double() - 127))
    return (v.view(rows, -1, 32) * factor[:, :, None]).view(rows, -1)[:, :cols]
