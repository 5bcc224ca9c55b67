"""8-bit floating point and the AdamW step from their definitions (include/gq.h), in torch and 64 bits, on any
device: codes and exponents bit for bit."""
import torch

import activation_ref

E4M3_MOST, ROOT_MOST = 448.0, 31.0 * 2 ** 14


def two(e):
    """2^e from its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exponents(top, most):
    """The smallest E >= 1 with most * 2^(E - 127) >= top, 255 where top is not finite."""
    bad = ~torch.isfinite(top)
    t = torch.where(bad, torch.zeros_like(top), top)
    mant, exp = torch.frexp(t)
    m, b = torch.frexp(torch.tensor(most, dtype=torch.float64, device=top.device))
    e = exp - b + (mant > m).to(exp.dtype) + 127
    e = torch.where(t == 0, torch.ones_like(e), e.clamp(min=1))
    return torch.where(bad, torch.full_like(e, 255), e).long()


def spacing(y, bits, low):
    """The distance of neighbours at y >= 0 among numbers of `bits` fraction bits, 2^low apart near 0."""
    exp = torch.frexp(y)[1]
    return two(torch.where(y == 0, torch.full_like(exp, low), (exp - 1 - bits).clamp(min=low)))


def fp8(x, block_rows):
    """(codes' values in units of the block's step, E per block) of a matrix."""
    x = x.double()
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % block_rows))
    v = v.reshape(v.shape[0] // block_rows, block_rows, -1, 128)
    a = v.abs()
    top = torch.where(torch.isfinite(a), a, torch.full_like(a, float("inf"))).amax(dim=(1, 3))
    e = exponents(top, E4M3_MOST)
    y = v / two(e - 127)[:, None, :, None]
    y = torch.where((e == 255)[:, None, :, None], torch.zeros_like(y), y)
    s = spacing(y.abs(), 3, -9)
    q = torch.round(y / s) * s
    return q.reshape(-1, q.shape[2] * 128)[:rows, :cols], e


def values(q, e, block_rows):
    """What fp8() stands for, NaN in marked blocks."""
    rows, cols = q.shape
    step = torch.where(e == 255, torch.full_like(e, 0).double() + float("nan"), two(e - 127))
    step = step.repeat_interleave(block_rows, dim=0).repeat_interleave(128, dim=1)
    return q * step[:rows, :cols]


def words(n, row, seed, step, device):
    """The 16-bit numbers of the first n columns of a row of the library's stream."""
    g = (n + 7) // 8
    import numpy as np
    i = np.arange(g, dtype=np.uint64)
    w = activation_ref.philox((i, np.full_like(i, row), np.full_like(i, step & 0xFFFFFFFF),
                               np.full_like(i, step >> 32)), (seed & 0xFFFFFFFF, seed >> 32))
    h = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], axis=1)
    return torch.from_numpy(h.reshape(-1)[:n].astype(np.int64)).to(device).double()


def on_grid(x, most, bits, low, h, keep):
    """x >= 0 rounded on the grids of its blocks of 32 (h: 16-bit numbers, or None for to nearest even); E per
    block; and the spacing of the grid at every element.  keep: what is not 0 does not become 0."""
    n = x.numel()
    v = torch.nn.functional.pad(x, (0, -n % 32)).view(-1, 32)
    top = torch.where(torch.isfinite(v), v, torch.full_like(v, float("inf"))).amax(1)
    e = exponents(top, most)
    unit = two(e - 127)[:, None]
    y = torch.where((e == 255)[:, None], torch.zeros_like(v), v / unit)
    s = spacing(y, bits, low)
    if h is None:
        q = torch.round(y / s) * s
    else:
        h = torch.nn.functional.pad(h, (0, -n % 32)).view(-1, 32)
        q = torch.floor(y / s + (h + 0.5) / 65536.0) * s
    if keep:
        q = torch.where((q == 0) & (y > 0), torch.full_like(q, 2.0 ** low), q)
    step = torch.where(e == 255, torch.full_like(top, float("nan")), two(e - 127))[:, None]
    return (q * step).view(-1)[:n], e, (s * unit).view(-1)[:n]


def adamw(p, g, m, v, step, lr, betas, eps, decay, clip=1.0):
    """(p, m, v) after a step, from the formulas."""
    p, g, m, v = p.double(), g.double() * clip, m.double(), v.double()
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    fix = (1 - b2 ** step) ** 0.5
    p = p * (1 - lr * decay) - lr / (1 - b1 ** step) * m / (v.sqrt() / fix + eps)
    return p, m, v
