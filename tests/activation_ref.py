"""The activation operators from their definitions (include/gq.h), in numpy and 64 bits: block
exponents and codes bit for bit, layer norm, GELU and the weight gradient."""
import math

import numpy as np

try:
    from scipy.special import erfc
except ImportError:  # the standard library's, element by element
    erfc = np.vectorize(math.erfc, otypes=[np.float64])

M32 = np.uint64(0xFFFFFFFF)


def philox(c, key):
    """Philox4x32-10: c is four arrays of counter words, key two numbers."""
    c = [np.asarray(v, dtype=np.uint64) for v in c]
    k = list(key)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & M32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def random16(rows, cols, seed, step):
    """The high 16 bits of every element's word."""
    g = (cols + 7) // 8
    i, j = np.meshgrid(np.arange(rows), np.arange(g), indexing="ij")
    w = philox((j, i, np.full_like(i, step & 0xFFFFFFFF), np.full_like(i, step >> 32)),
               (seed & 0xFFFFFFFF, seed >> 32))
    h = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], axis=2)
    return h.reshape(rows, g * 8)[:, :cols].astype(np.int64)


def pitches(cols):
    p = (cols + 31) // 32 * 32
    return p, (p // 32 + 15) // 16 * 16


def quantise(x, seed=None, step=0):
    """(codes rows x pitch, exps rows x blocks) of a float matrix."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    pitch = pitches(cols)[0]
    v = np.zeros((rows, pitch))
    v[:, :cols] = x
    blocks = v.reshape(rows, -1, 32)
    top = np.abs(blocks).max(axis=2)  # NaN stays NaN
    bad = ~(top <= 127.0 * 2.0 ** 121)
    t = np.where(bad, 0.0, top)
    mant, ex = np.frexp(t)  # t = mant 2^ex, mant in [1/2, 1)
    e = np.where(mant <= 127 / 128, ex - 7, ex - 6) + 127
    e = np.where(t == 0, 1, np.maximum(e, 1))
    unit = np.ldexp(1.0, e - 127)
    with np.errstate(invalid="ignore"):
        q = np.where(bad[:, :, None], 0.0, blocks / unit[:, :, None]).reshape(rows, pitch)
    if seed is None:
        codes = np.rint(q)
    else:
        p = 2 * np.rint(q * 32768.0)
        p[:, :cols] += random16(rows, cols, seed, step)
        codes = np.floor(p / 65536.0)
    return codes.astype(np.int8), np.where(bad, 255, e).astype(np.uint8)


def values(codes, exps, cols):
    rows = codes.shape[0]
    blocks = codes.shape[1] // 32
    e = exps[:, :blocks].astype(np.int64)
    unit = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    v = codes.astype(np.float64).reshape(rows, blocks, 32) * unit[:, :, None]
    return v.reshape(rows, -1)[:, :cols]


def layernorm(x, w, b, eps):
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    hat = d * rstd[:, None]
    return hat * w + b, mean, rstd, hat


def layernorm_backward(dy, w, rstd, hat):
    g = dy * w
    c1 = g.mean(axis=1, keepdims=True)
    c2 = (g * hat).mean(axis=1, keepdims=True)
    return rstd[:, None] * (g - c1 - hat * c2), (dy * hat).sum(axis=0), dy.sum(axis=0)


def gelu(u, form):
    """gelu and its derivative."""
    if form == "tanh":
        k, b = math.sqrt(2 / math.pi), 0.044715
        c = np.clip(u, -40, 40)
        t = np.tanh(k * (c + b * c ** 3))
        p = 1.0 / (1.0 + np.exp(-2 * k * (c + b * c ** 3)))
        return u * p, p + 0.5 * u * (1 - t * t) * k * (1 + 3 * b * c * c)
    p = 0.5 * erfc(-u / math.sqrt(2))
    with np.errstate(under="ignore", over="ignore"):
        phi = np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return u * p, p + u * phi
