"""Operators of a training step in few bits next to its 8-bit activations and compressed gradients: the
linear layers' products in 8-bit floating point, forward and for the input's gradient, and the AdamW step
over all parameters at once, as cases to measure.

A matrix in 8-bit floating point holds e4m3 codes (rows of round_up(cols, 16) bytes) and an exponent byte E
for each block of 128 columns of a row, or of 128 x 128 elements (weights): an element stands for
code * 2^(E - 127), E the smallest value >= 1 with 448 * 2^(E - 127) >= the block's largest magnitude.
Exponents lie as the tensor cores read them: [rows / 128][blocks / 4][32][4][4], the byte at [t][w][r][j][b]
is that of row 128 t + 32 j + r and block 4 w + b.

Optimizer states in 8 bits hold, for every 32 elements of a tensor, an exponent for the first moment (e4m3
codes, as above) and one for the root of the second: unsigned codes of 4 exponent and 4 fraction bits, in
units of 2^(E - 127), E the smallest value >= 1 with 31 * 2^14 * 2^(E - 127) >= the largest; a root that is
not zero keeps a code that is not zero.  Rounding is to nearest even, or at random without bias, with the
16-bit numbers of the library's Philox4x32-10 stream (key = seed, counter = element / 8, 3 t + k, step; t
the tensor, k = 0 for the first moment, 1 for the second, 2 for bf16 parameters).

own = False computes every operator from elementary torch operations in 32 bits; own = True calls the
library.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BETA1, BETA2, EPS, LR, DECAY, MAX_NORM = 0.9, 0.999, 1e-8, 1e-3, 0.01, 1.0


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # the step of a model of two narrow blocks, gradients clipped: latency counts
        dict(name="adamw_small_f32", op="adamw", layers=2, width=256, hidden=1024, param="f32", grad="f32",
             state="f32", random=False),
        # all MLP blocks of a 24-layer encoder, full-precision states, gradients clipped
        dict(name="adamw_large_f32", op="adamw", layers=24, width=1024, hidden=4096, param="f32",
             grad="f32", state="f32", random=False),
        # a narrow model of odd sizes kept in bf16, states in 8 bits
        dict(name="adamw_small_8bit", op="adamw", layers=3, width=250, hidden=1001, param="bf16",
             grad="bf16", state="8bit", random=True),
        # the 24-layer encoder again with states in 8 bits, rounded without bias
        dict(name="adamw_large_8bit", op="adamw", layers=24, width=1024, hidden=4096, param="f32",
             grad="bf16", state="8bit", random=True),
        # a weight after its step, for the next forward and backward pass
        dict(name="fp8_weight", op="fp8", rows=4096, cols=4096, dtype="f32", tiles=True),
        # the activations of a large micro-batch
        dict(name="fp8_rows_large", op="fp8", rows=32768, cols=4096, dtype="bf16", tiles=False),
        # one token through a 4096-wide layer
        dict(name="linear_token", op="linear", rows=1, cols=4096, outs=4096, dtype="bf16", out="bf16",
             bias=False),
        # a projection over one sequence
        dict(name="linear_small", op="linear", rows=384, cols=768, outs=768, dtype="bf16", out="bf16",
             bias=True),
        # full-precision activations of a width that fits no block
        dict(name="linear_odd_f32", op="linear", rows=1021, cols=1001, outs=2050, dtype="f32", out="f32",
             bias=True),
        # a 4096-wide layer over a long batch
        dict(name="linear_large", op="linear", rows=16384, cols=4096, outs=4096, dtype="bf16", out="bf16",
             bias=True),
        # the gradient of one short sequence behind a narrow layer
        dict(name="dgrad_small", op="dgrad", rows=100, cols=256, outs=1024, dtype="bf16", out="bf16"),
        # the gradient of a long batch behind a layer that widens
        dict(name="dgrad_large", op="dgrad", rows=16384, cols=1024, outs=4096, dtype="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; a multiple of 64 half of the time where it is large enough."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if v >= 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["adamw", "adamw", "fp8", "linear", "linear", "dgrad"])
    if op == "adamw":
        state = rng.choice(["f32", "8bit"])
        param = rng.choice(["f32", "f32", "bf16"])
        return dict(op=op, layers=_log(rng, 1, 24), width=_size(rng, 16, 1024), hidden=_size(rng, 16, 4096),
                    param=param, grad="bf16" if param == "bf16" else rng.choice(["f32", "bf16"]),
                    state=state, random=(state == "8bit" or param == "bf16") and rng.random() < 0.7)
    if op == "fp8":
        cols = _size(rng, 16, 8192)
        return dict(op=op, rows=_size(rng, 1, min(32768, (1 << 27) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]), tiles=rng.random() < 0.4)
    cols, outs = _size(rng, 16, 8192), _size(rng, 16, 8192)
    if op == "dgrad":  # its sums run over outs
        c = dict(op=op, cols=cols, outs=outs)
    else:
        c = dict(op=op, cols=cols, outs=outs, bias=rng.random() < 0.5)
    c["rows"] = _size(rng, 1, min(16384, (1 << 38) // (cols * outs)))
    c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    c["out"] = "bf16" if c["dtype"] == "bf16" else rng.choice(["f32", "bf16"])
    return c


def _bytes(t):
    return 4 if t == "f32" else 2


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(a * b for a, b in _shapes(case))
        fixed = 2 * _bytes(case["param"]) + _bytes(case["grad"])
        if case["state"] == "f32":
            return {"bytes": n * (fixed + 16), "flops": 18 * n}
        # codes and exponents read and written, and their values given back in bf16
        return {"bytes": int(n * (fixed + 4 + 4 / 32 + 4)), "flops": 40 * n}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if op == "fp8":
        codes = n + (n // 16384 if case["tiles"] else n // 128)
        return {"bytes": n * (_bytes(case["dtype"]) + 2) + 2 * codes, "flops": 4 * n}
    outs = case["outs"]
    weight = outs * cols + outs * cols // 16384
    if op == "linear":
        move = n * _bytes(case["dtype"]) + rows * outs * _bytes(case["out"]) + (4 * outs if case["bias"] else 0)
    else:
        move = rows * outs * _bytes(case["dtype"]) + n * _bytes(case["out"])
    return {"bytes": weight + move, "flops": 2 * n * outs}


# ---- inputs --------------------------------------------------------------------------------

def _shapes(case):
    """The parameters of MLP blocks: norm weight and bias, and two linear layers with their biases."""
    w, h = case["width"], case["hidden"]
    return [(1, w), (1, w), (h, w), (1, h), (w, h), (1, w)] * case["layers"]


def _up(v, m):
    return (v + m - 1) // m * m


def _lay_out(blocks):
    """An exponent byte per row and block as the tensor cores read them."""
    rows, n = blocks.shape
    e = torch.ones((_up(rows, 128), _up(n, 4)), dtype=torch.uint8, device=blocks.device)
    e[:rows, :n] = blocks
    return e.view(-1, 4, 32, e.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _activations(g, rows, cols, dtype):
    """Normal values with channels of unequal scale, a few strong ones, and padding rows of zeros."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    scale = torch.exp(0.3 * torch.randn(cols, generator=g, device="cuda"))
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 4.0 * scale, scale)
    if rows >= 32:
        x[-(rows // 32):] = 0.0
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case, seed=seed * 2654435761 % (1 << 63), step=1 + seed % 1000)
    if op == "adamw":
        return _prepare_adamw(case, g, s)
    dtype, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
    if op == "fp8":
        s["x"] = _activations(g, rows, cols, dtype)
        return s
    outs = case["outs"]
    w = torch.randn((outs, cols), generator=g, device="cuda") * cols ** -0.5
    w *= torch.exp(0.2 * torch.randn((outs, 1), generator=g, device="cuda"))
    # the weight that a program keeps: codes, and its 128 x 128 blocks' exponents for either product
    codes, e = _quantise(w, True)
    s["codes"], s["e"] = codes, e
    s["exps"] = _lay_out(e.repeat_interleave(128, dim=0)[:outs])
    s["exps_t"] = _lay_out(e.t().repeat_interleave(128, dim=0)[:cols])
    if op == "linear":
        s["x"] = _activations(g, rows, cols, dtype)
        s["bias"] = 0.1 * torch.randn(outs, generator=g, device="cuda") if case["bias"] else None
    else:
        dy = torch.randn((rows, outs), generator=g, device="cuda") * 1e-3
        dy *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
        if rows >= 32:
            dy[-(rows // 32):] = 0.0
        s["dy"] = dy.to(dtype)
    return s


def _prepare_adamw(case, g, s):
    shapes = _shapes(case)
    numel = [a * b for a, b in shapes]
    room = [_up(n, 32) for n in numel]  # each tensor begins at a multiple of 32 of one buffer
    total = sum(room)
    at = [sum(room[:i]) for i in range(len(room))]
    real = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(at, numel):
        real[a:a + n] = True

    def normal(spread, dtype=torch.float32):
        x = torch.randn(total, generator=g, device="cuda") * spread
        return torch.where(real, x, 0.0).to(dtype)

    # clipped where the states are fp32, below the limit otherwise
    size = (3.0 if case["state"] == "f32" else 0.3) / math.sqrt(sum(numel))
    p, grad = normal(0.02, DTYPES[case["param"]]), normal(size, DTYPES[case["grad"]])
    m = normal(0.3 * size)
    v = torch.where(real, normal(0.5).exp() * (size * size), 0.0)
    s.update(p=p, grad=grad, numel=numel, room=room)

    def cut(x):
        return [t[:n].view(shape) for t, n, shape in zip(x.split(room), numel, shapes)]

    s["params"], s["grads"] = cut(p), cut(grad)
    if case["state"] == "f32":
        s.update(m=m, v=v)
        s["states"] = list(zip(cut(m), cut(v)))
    else:
        cm, em = _moment_codes(m, None)
        cv, ev = _root_codes(v.sqrt(), None)
        s.update(cm=cm, cv=cv, exps=torch.stack((em, ev), dim=1).contiguous())
        s["states"] = list(zip(cm.split(room), cv.split(room), s["exps"].split([r // 32 for r in room])))
    return s


# ---- the plain forms -----------------------------------------------------------------------

def _quantise(x, tiles):
    """e4m3 codes (rows of round_up(cols, 16) bytes) and exponents, one per 128 columns of a row or per
    128 x 128 elements."""
    rows, cols = x.shape
    high, wide = _up(rows, 128) if tiles else rows, _up(cols, 128)
    v = torch.zeros((high, wide), device=x.device)
    v[:rows, :cols] = x
    r = 128 if tiles else 1
    v = v.view(high // r, r, wide // 128, 128)
    top = v.abs().amax(dim=(1, 3)).view(torch.int32)
    e = (((top + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    v = v * ((254 - e) << 23).view(torch.float32)[:, None, :, None]  # times 2^(127 - E), exact
    codes = v.view(high, wide)[:rows, :_up(cols, 16)].to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), e.to(torch.uint8)


def _values(codes, e, cols):
    """What codes and exponents stand for, in fp32."""
    rows = codes.shape[0]
    step = (e.to(torch.int32) << 23).view(torch.float32)
    step = step.repeat_interleave(128, dim=1)[:, :cols]
    if e.shape[0] != rows:
        step = step.repeat_interleave(128, dim=0)[:rows]
    return codes[:, :cols].view(torch.float8_e4m3fn).float() * step


def _words(group, row, seed, step):
    """The 16-bit numbers of the groups of 8 elements, in order."""
    low = 0xFFFFFFFF
    c0, c1 = group, row
    c2 = torch.full_like(c0, step & low)
    c3 = torch.full_like(c0, step >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products, kept modulo 2^64
        c0, c1, c2, c3 = (((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), dim=1)
    return torch.stack((words & 0xFFFF, words >> 16), dim=2).view(-1).to(torch.int32)


def _groups(room):
    """Of every group of 8 elements of the buffer: its place in its tensor, and that tensor's number."""
    count = torch.tensor([r // 8 for r in room], device="cuda")
    n = sum(room) // 8
    owner = torch.repeat_interleave(torch.arange(len(room), device="cuda"), count, output_size=n)
    return torch.arange(n, device="cuda") - (count.cumsum(0) - count)[owner], owner


def _round_bits(bits, drop, h):
    """Bits rounded off at the right, to nearest even or with 16-bit numbers."""
    if h is None:
        return (bits + ((1 << (drop - 1)) - 1) + ((bits >> drop) & 1)) >> drop
    return (bits + ((h << (drop - 16)) | (1 << (drop - 17)))) >> drop


def _scale(e):
    return (e << 23).view(torch.float32)[:, None]


def _moment_codes(m, h):
    v = m.view(-1, 32)
    e = (((v.abs().amax(1).view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    y = (v.abs() * _scale(254 - e)) * 2.0 ** -120  # e4m3's exponent field becomes fp32's
    code = _round_bits(y.view(torch.int32), 20, None if h is None else h.view(-1, 32))
    code = code | torch.where(v < 0, 128, 0)
    return code.to(torch.uint8).view(-1), e.to(torch.uint8)


def _moment_values(codes, e):
    v = codes.view(torch.float8_e4m3fn).float().view(-1, 32)
    return (v * _scale(e.to(torch.int32))).view(-1)


def _root_codes(r, h):
    v = r.view(-1, 32)
    e = (((v.amax(1).view(torch.int32) + 0x7FFFF) >> 23) - 18).clamp(min=1)
    y = (v * _scale(188 - e)) * 2.0 ** -64  # in units of 2^-130: 4 bits behind the exponent field
    code = _round_bits(y.view(torch.int32), 19, None if h is None else h.view(-1, 32))
    code = torch.maximum(code, (v > 0).to(torch.int32))
    return code.to(torch.uint8).view(-1), e.to(torch.uint8)


def _root_values(codes, e):
    v = (codes.to(torch.int32) << 19).view(torch.float32).view(-1, 32) * 2.0 ** 64
    return (v * _scale(e.to(torch.int32) + 66)).view(-1)


def _plain_adamw(s):
    case = s["case"]
    eight, rnd = case["state"] == "8bit", case["random"]
    grad = s["grad"].float()
    norm = grad.square().sum().sqrt()
    grad = grad * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    if eight:
        m = _moment_values(s["cm"], s["exps"][:, 0])
        v = _root_values(s["cv"], s["exps"][:, 1]).square()
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + grad * (1.0 - BETA1)
    v = v * BETA2 + grad.square() * (1.0 - BETA2)
    root = v.sqrt()
    t = s["step"]
    size, fix = LR / (1.0 - BETA1 ** t), 1.0 / math.sqrt(1.0 - BETA2 ** t)
    p = s["p"].float() * (1.0 - LR * DECAY) - m / (root * fix + EPS) * size
    if rnd:
        at, owner = _groups(s["room"])
    if case["param"] == "bf16" and rnd:
        h = _words(at, 3 * owner + 2, s["seed"], t)
        p = ((p.view(torch.int32) + h) & -65536).view(torch.float32)
    s["p"].copy_(p)
    out = [norm.view(1), s["p"]]
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return out + [s["m"], s["v"]]
    cm, em = _moment_codes(m, _words(at, 3 * owner, s["seed"], t) if rnd else None)
    cv, ev = _root_codes(root, _words(at, 3 * owner + 1, s["seed"], t) if rnd else None)
    s["cm"].copy_(cm)
    s["cv"].copy_(cv)
    s["exps"].copy_(torch.stack((em, ev), dim=1))
    return out + [_moment_values(cm, em).to(torch.bfloat16), _root_values(cv, ev).to(torch.bfloat16)]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        return _plain_adamw(s)
    cols = case["cols"]
    if op == "fp8":
        return _values(*_quantise(s["x"].float(), case["tiles"]), cols).to(torch.bfloat16)
    w = _values(s["codes"], s["e"], cols)
    if op == "linear":
        y = _values(*_quantise(s["x"].float(), False), cols) @ w.t()
        return (y if s["bias"] is None else y + s["bias"]).to(DTYPES[case["out"]])
    return (_values(*_quantise(s["dy"].float(), False), case["outs"]) @ w).to(DTYPES[case["out"]])


# ---- the library ---------------------------------------------------------------------------

def _cut(x, s):
    """The tensors' elements of a buffer, without what lies behind them in their room."""
    sizes = [v for n, room in zip(s["numel"], s["room"]) for v in ((n, room - n) if n < room else (n,))]
    gap = [k for n, room in zip(s["numel"], s["room"]) for k in ((False, True) if n < room else (False,))]
    return [t for t, k in zip(x.split(sizes), gap) if not k]


def _library(s):
    import allreduce_compatible_gradient_gb300 as gq

    case = s["case"]
    op = case["op"]
    if op == "adamw":
        eight = case["state"] == "8bit"
        states = [gq.Adam8(*t) for t in s["states"]] if eight else s["states"]
        norm = gq.gq_tensors_norm(s["grads"])
        gq.gq_adamw_step(s["params"], s["grads"], states, s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                         weight_decay=DECAY, norm=norm, max_norm=MAX_NORM,
                         seed=s["seed"] if case["random"] else None)
        if not eight:
            return [norm, s["p"], s["m"], s["v"]]
        # the states' values, in one buffer like the parameters
        new = torch.empty if s["numel"] == s["room"] else torch.zeros
        m, r = (new(sum(s["room"]), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gq.gq_adamw_values(states, out=(_cut(m, s), _cut(r, s)))
        return [norm, s["p"], m, r]
    if op == "fp8":
        return gq.gq_fp8_dequantize(gq.gq_fp8_quantize(s["x"], tiles=case["tiles"]),
                                    out_dtype=torch.bfloat16)
    weight = gq.Fp8(s["codes"], s["exps"], case["cols"], exps_t=s["exps_t"])
    if op == "linear":
        return gq.gq_fp8_linear(s["x"], weight, bias=s["bias"], out_dtype=DTYPES[case["out"]])
    return gq.gq_fp8_linear_dgrad(s["dy"], weight, out_dtype=DTYPES[case["out"]])


def run(state):
    return _library(state) if own else _plain(state)


# ---- 64-bit results ------------------------------------------------------------------------

def _two(e):
    """2^e, put together from its exponent field: pow() is not exact in 64 bits on the GPU."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _least(top, most):
    """The smallest j >= -126 with most * 2^j >= top."""
    mant, exp = torch.frexp(top)
    base = math.frexp(most)
    j = exp - base[1] + (mant > base[0]).to(exp.dtype)
    return torch.where(top == 0, torch.full_like(j, -126), j.clamp(min=-126))


def _grid(y, bits, low):
    """The spacing at y >= 0 of numbers with `bits` fraction bits whose least spacing is 2^low."""
    exp = torch.frexp(y)[1]
    return _two(torch.where(y == 0, torch.full_like(exp, low), (exp - 1 - bits).clamp(min=low)))


def _exact_rows(x, tiles):
    rows, cols = x.shape
    out = torch.empty_like(x)
    step = 128 if tiles else 2048
    for r in range(0, rows, step):
        v = torch.nn.functional.pad(x[r:r + step], (0, -cols % 128))
        v = v.reshape(v.shape[0], -1, 128)
        top = v.abs().amax(dim=2)
        unit = _two(_least(top.amax(0, keepdim=True) if tiles else top, 448.0))[:, :, None]
        y = v / unit
        s = _grid(y.abs(), 3, -9)
        out[r:r + step] = (torch.round(y / s) * s * unit).reshape(v.shape[0], -1)[:, :cols]
    return out


def _mulhilo(a, m):
    """High and low 32 bits of a * m, from 16-bit limbs."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a1 * m0 + ((a0 * m0) >> 16)
    mid2 = (mid & 0xFFFF) + a0 * m1
    return a1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((a0 * m0) & 0xFFFF)


def _exact_words(n, row, seed, step):
    """The 16-bit numbers of a tensor's first n elements, in a row of the stream."""
    g = torch.arange(_up(n, 8) // 8, device="cuda")
    w = [g, torch.full_like(g, row), torch.full_like(g, step % 2 ** 32), torch.full_like(g, step // 2 ** 32)]
    for r in range(10):
        h0, l0 = _mulhilo(w[0], 0xD2511F53)
        h1, l1 = _mulhilo(w[2], 0xCD9E8D57)
        w = [h1 ^ w[1] ^ ((seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32), l1,
             h0 ^ w[3] ^ ((seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32), l0]
    halves = [v for word in w for v in (word % 65536, word // 65536)]
    return torch.stack(halves, dim=1).reshape(-1)[:n].double()


def _exact_round(x, most, bits, low, u):
    """x >= 0 on the grid of its blocks of 32, to nearest or at random."""
    n = x.numel()
    v = torch.nn.functional.pad(x, (0, -n % 32)).view(-1, 32)
    unit = _two(_least(v.amax(1), most))[:, None]
    y = v / unit
    s = _grid(y, bits, low)
    k = torch.round(y / s) if u is None else torch.floor(
        y / s + (torch.nn.functional.pad(u, (0, -n % 32)).view(-1, 32) + 0.5) / 65536.0)
    return s * k * unit, v, s * unit


def _exact_adamw(case, s):
    total = sum(s["room"])
    outs = [torch.zeros(total, dtype=torch.float64, device="cuda") for _ in range(3)]
    grads = [t.double().reshape(-1) for t in s["grads"]]
    norm = torch.stack([torch.dot(t, t) for t in grads]).sum().sqrt()
    clip = min(1.0, MAX_NORM / (float(norm) + 1e-6))
    t, at = s["step"], 0
    for i, (grad, param, state) in enumerate(zip(grads, s["params"], s["states"])):
        n = grad.numel()
        grad = grad * clip
        if case["state"] == "f32":
            m, v = (x.double().reshape(-1) for x in state)
        else:
            unit = _two(state[2].int() - 127).repeat_interleave(32, dim=0)[:n]
            m = state[0][:n].view(torch.float8_e4m3fn).double() * unit[:, 0]
            c = state[1][:n].long()
            v = torch.where(c < 16, c, (16 + c % 16) << (c // 16 - 1).clamp(min=0)).double() * unit[:, 1]
            v = v * v
        m = torch.lerp(grad, m, BETA1)
        v = torch.lerp(grad * grad, v, BETA2)
        root = torch.sqrt(v)
        step = (m / (1.0 - BETA1 ** t)) / (root / math.sqrt(1.0 - BETA2 ** t) + EPS)
        p = param.double().reshape(-1)
        p = p - LR * DECAY * p - LR * step
        words = [None] * 3
        if case["random"]:
            words = [_exact_words(n, 3 * i + k, s["seed"], t) for k in range(3)]
        if case["param"] == "bf16" and words[2] is not None:
            unit = _grid(p.abs(), 7, -133)
            p = torch.sign(p) * torch.floor(p.abs() / unit + words[2] / 65536.0) * unit
        if case["state"] == "8bit":
            q, _, _ = _exact_round(m.abs(), 448.0, 3, -9, words[0])
            m = torch.sign(m) * q.view(-1)[:n]
            q, r, unit = _exact_round(root, 31.0 * 2 ** 14, 4, 0, words[1])
            v = torch.where((q == 0) & (r > 0), unit, q).view(-1)[:n]
        for o, x in zip(outs, (p, m, v)):
            o[at:at + n] = x
        at += s["room"][i]
    return [norm.view(1)] + outs


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(case, s)
    if op == "fp8":
        return _exact_rows(s["x"].double(), case["tiles"])
    n = -(-case["cols"] // 128)
    unit = _two(s["e"].int() - 127)[:, :n].repeat_interleave(128, dim=1).repeat_interleave(128, dim=0)
    w = s["codes"][:, :case["cols"]].view(torch.float8_e4m3fn).double()
    w = w * unit[:w.shape[0], :w.shape[1]]
    if op == "dgrad":
        return torch.mm(_exact_rows(s["dy"].double(), False), w)
    y = torch.nn.functional.linear(_exact_rows(s["x"].double(), False), w)
    return y if s["bias"] is None else y + s["bias"].double()
