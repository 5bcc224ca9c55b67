"""The activation operators on the GPU against their definitions in 64 bits.

Tolerances, with u = 2^-24 (half a unit in the last place of fp32) and 2^-9 of bf16's:
- codes and exponents are exact: every operation they depend on is exact or defined to round once;
- a sum of n terms added in any order is within n u of the sum of their magnitudes;
- the tensor cores add 16 products at a time and may truncate, 2^-22 of the largest partial sum a
  time: within (n / 16 + 32) 2^-22 of the sum of the magnitudes;
- an elementwise fp32 formula of k operations is within 2 k u of the magnitudes it adds up; the
  exponential and reciprocal of the hardware are within 4 u, the polynomials within 1.5e-7 (fp32)
  or 5e-6 (bf16).
"""
import numpy as np
import pytest

import activation_ref as ref
from gpu_common import gq_module

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def gq():
    return gq_module()


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


DT = ["f32", "bf16"]


def types(torch, name):
    return torch.float32 if name == "f32" else torch.bfloat16


def tensor(torch, a, dtype, extra=0):
    """a on the GPU as dtype, rows extra elements further apart than their length; and its values."""
    t = torch.empty((a.shape[0], a.shape[1] + extra), dtype=types(torch, dtype), device="cuda")
    t.fill_(float("nan"))
    t = t[:, :a.shape[1]]
    t.copy_(torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)))
    return t, host(t)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(rows, cols, seed, scale=1.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)) * np.exp(r.standard_normal((1, cols)))
    if rows > 2:
        x[rows // 2] = 0.0          # a padding row
    if cols > 40:
        x[0, 32:64] = 0.0           # a block of zeros
    return x * scale


def checkpoint(gq, torch, x, **kw):
    act = gq.gq_act_quantize(x, **kw)
    return act, act.codes.cpu().numpy(), act.exps.cpu().numpy()


def near(got, want, tol, dtype):
    """|got - want| <= tol (+ the rounding of bf16), NaN where want is NaN."""
    assert got.shape == want.shape
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    ok = ~bad & ~inf
    tol = np.broadcast_to(tol, want.shape)[ok] + (2.0 ** -8 * np.abs(want[ok]) if dtype == "bf16"
                                                  else U * np.abs(want[ok])) + 1e-37
    d = np.abs(got[ok] - want[ok])
    assert (d <= tol).all(), (d.max(), (d / tol).max())


# more rows than two per SM: several rows at a time per block (one to four warps each), and one row of
# up to 16 warps
WALKED = [(400, 512), (700, 1024), (320, 768), (350, 4096), (310, 8192), (400, 200)]

SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 7), (33, 100), (4, 255), (9, 256), (7, 257),
          (17, 512), (3, 1000), (130, 768), (19, 1024), (2, 1025), (5, 2048), (3, 4100), (2, 8192),
          (1, 8200), (2, 17000), (1, 40001)]


@pytest.mark.parametrize("extra", [0, 3, 8, 16])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_checkpoint_codes_are_exact(gq, torch, rows, cols, dtype, extra):
    x, xv = tensor(torch, inputs(rows, cols, rows * cols), dtype, extra)
    for kw in (dict(), dict(seed=0x1234567890ABCDEF, step=(5 << 32) + 77)):
        act, codes, exps = checkpoint(gq, torch, x, **kw)
        wc, we = ref.quantise(xv, kw.get("seed"), kw.get("step", 0))
        assert np.array_equal(exps[:, :we.shape[1]], we)
        assert np.array_equal(codes, wc)
        want = ref.values(wc, we, cols)
        for out_dtype in (torch.float32, torch.bfloat16):
            got = gq.gq_act_dequantize(act, out_dtype=out_dtype)
            assert np.array_equal(host(got), want)


@pytest.mark.parametrize("dtype", DT)
def test_checkpoint_of_special_values(gq, torch, dtype):
    """Blocks with an infinity or a NaN read back as NaN, their neighbours as themselves; largest
    and smallest magnitudes, and the exponent's edge 127 / 64."""
    x = np.zeros((12, 100), dtype=np.float32)
    x[:] = np.linspace(-2, 2, 100)
    x[0, 5], x[1, 40], x[2, 99] = np.inf, np.nan, -np.inf
    x[3, :] = 127 / 64
    x[4, :] = np.nextafter(np.float32(127 / 64), np.float32(4))
    x[5, :] = 3.0e38
    x[6, 0] = 3.3895314e38      # bf16's largest: above 127 * 2^121
    x[7, :] = 1e-38
    x[8, :] = 2.0 ** -130       # denormal: below half the smallest step
    x[9, ::2] *= 1e-30
    x[10, :] = -127 / 64
    x[11, :] = 2.0 ** -126 * 126.6
    t, xv = tensor(torch, x, dtype)
    for kw in (dict(), dict(seed=3, step=1)):
        act, codes, exps = checkpoint(gq, torch, t, **kw)
        wc, we = ref.quantise(xv, kw.get("seed"), kw.get("step", 0))
        assert np.array_equal(exps[:, :4], we) and np.array_equal(codes, wc)
        got, want = host(gq.gq_act_dequantize(act, out_dtype=torch.float32)), ref.values(wc, we, 100)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_random_rounding_is_unbiased(gq, torch):
    """Mean over many steps within 5 standard errors of the value; each rounding is one of the two
    neighbouring levels."""
    x = np.linspace(-1.9, 1.9, 96).reshape(1, 96)
    t, xv = tensor(torch, x, "f32")
    n, total = 400, np.zeros_like(xv)
    for step in range(n):
        v = host(gq.gq_act_dequantize(gq.gq_act_quantize(t, seed=11, step=step),
                                      out_dtype=torch.float32))
        assert (np.abs(v - xv) < 2.0 ** -6 + 1e-12).all()
        total += v
    assert (np.abs(total / n - xv) < 5 * 2.0 ** -7 / np.sqrt(n)).all()


def test_half_output_rounds(gq, torch):
    x, xv = tensor(torch, inputs(4, 64, 1, 1e5), "f32")
    act, codes, exps = checkpoint(gq, torch, x)
    want = ref.values(codes, exps, 64).astype(np.float32).astype(np.float16)
    got = gq.gq_act_dequantize(act, out_dtype=torch.float16).cpu().numpy()
    assert np.array_equal(got, want)


# ---- layer norm ----------------------------------------------------------------------------

def affine(torch, cols, kind, seed):
    r = np.random.default_rng(seed)
    w, b = 1 + 0.3 * r.standard_normal(cols), 0.5 * r.standard_normal(cols)
    if kind == "none":
        return None, None, np.ones(cols), np.zeros(cols)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    wt, bt = (torch.tensor(v, dtype=torch.float32).to(t).cuda() for v in (w, b))
    return wt, bt, host(wt), host(bt)


@pytest.mark.parametrize("extra,kind", [(0, "f32"), (3, "bf16"), (8, "none")])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", SHAPES + WALKED)
def test_layernorm_forward(gq, torch, rows, cols, dtype, extra, kind):
    x, xv = tensor(torch, inputs(rows, cols, 3 * rows + cols) + 0.7, dtype, extra)
    w, b, wv, bv = affine(torch, cols, kind, cols)
    y, mean, rstd, act = gq.gq_layernorm_forward(x, w, b, eps=1e-5, seed=9, step=4)
    wy, wm, wr, hat = ref.layernorm(xv, wv, bv, 1e-5)
    size = np.abs(xv).mean(axis=1)
    near(host(mean), wm, (cols + 2) * U * size, "f32")
    # d = x - mean is off by the mean's error and its own rounding; the variance by twice that
    dm = ((cols + 2) * U * size + U * np.abs(xv).max(axis=1)) * wr
    rel = (cols + 8) * U + 2 * dm
    near(host(rstd), wr, rel * wr, "f32")
    toly = np.abs(hat * wv) * (rel[:, None] + 4 * U) + np.abs(wv) * dm[:, None] + 2 * U * np.abs(bv)
    near(host(y), wy, toly, dtype)
    # the checkpoint is that of the fp32 normalised row: a code moves by one where the last bits
    # of the row cross a rounding boundary
    wc, we = ref.quantise(hat, 9, 4)
    exps, codes = act.exps.cpu().numpy()[:, :we.shape[1]], act.codes.cpu().numpy()
    # (a block whose values are all within their own error of 0, a constant row's, says nothing
    # about the exponent)
    err = np.abs(hat) * (rel[:, None] + 2 * U) + dm[:, None]
    block = lambda a: np.pad(a, ((0, 0), (0, -cols % 32))).reshape(rows, -1, 32).max(axis=2)  # noqa: E731
    sound = block(np.abs(hat)) > 1000 * block(err)
    assert (exps == we)[sound].mean() > 0.98 if sound.any() else True
    same = np.repeat((exps == we) & sound, 32, axis=1)
    assert np.abs(codes.astype(int) - wc)[same].max(initial=0) <= 1
    step = np.ldexp(1.0, exps.astype(int) - 127).repeat(32, axis=1)[:, :cols]
    assert (np.abs(ref.values(codes, exps, cols) - hat) <= step + err).all()
    assert not codes[:, cols:].any()
    y2, _, _, none = gq.gq_layernorm_forward(x, w, b, checkpoint=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("source", ["codes", "input"])
@pytest.mark.parametrize("extra,kind,gtype", [(0, "f32", "f32"), (3, "bf16", "bf16"), (8, "none", "f32")])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", SHAPES + WALKED + [(700, 96), (333, 1030), (300, 9000)])
def test_layernorm_backward(gq, torch, rows, cols, dtype, extra, kind, gtype, source):
    x, xv = tensor(torch, inputs(rows, cols, 5 * rows + cols) + 0.3, dtype, extra)
    dy, dyv = tensor(torch, inputs(rows, cols, 7 * rows + cols, 1e-2), dtype, extra)
    w, b, wv, _ = affine(torch, cols, kind, cols)
    _, mean, rstd, act = gq.gq_layernorm_forward(x, w, b)
    rv = host(rstd)
    if source == "codes":
        got = gq.gq_layernorm_backward(dy, w, rstd, act=act, grad_dtype=types(torch, gtype))
        hat = ref.values(act.codes.cpu().numpy(), act.exps.cpu().numpy(), cols)
        off = 0.0
    else:
        got = gq.gq_layernorm_backward(dy, w, rstd, x=x, mean=mean, grad_dtype=types(torch, gtype))
        hat = (xv - host(mean)[:, None]) * rv[:, None]
        off = 2 * U * (np.abs(xv) * rv[:, None] + np.abs(hat))
    wx, ww, wb = ref.layernorm_backward(dyv, wv, rv, hat)
    g = np.abs(dyv * wv)
    m1 = g.mean(axis=1, keepdims=True)
    m2 = (g * (np.abs(hat) + off)).mean(axis=1, keepdims=True)
    n = (cols + 8) * U
    tol = rv[:, None] * (4 * U * g + n * m1 + (np.abs(hat) + off) * n * m2 + off * m2 +
                         np.abs(hat) * (g * off).mean(axis=1, keepdims=True) + 4 * U * (m1 + np.abs(hat) * m2))
    near(host(got[0]), wx, tol, dtype)
    n = (rows + 40) * U
    near(host(got[1]), ww, n * (np.abs(dyv) * (np.abs(hat) + off)).sum(axis=0) +
         (np.abs(dyv) * off).sum(axis=0), gtype)
    near(host(got[2]), wb, n * np.abs(dyv).sum(axis=0), gtype)


def test_layernorm_gradients_against_differences(gq, torch):
    """dx, dw, db of the loss sum(y r) against central differences in 64 bits."""
    rows, cols, h = 3, 40, 1e-5
    r = np.random.default_rng(0)
    x0, w0, b0, g0 = (r.standard_normal(s) for s in ((rows, cols), cols, cols, (rows, cols)))
    x, xv = tensor(torch, x0, "f32")
    g, gv = tensor(torch, g0, "f32")
    w = torch.tensor(w0, dtype=torch.float32).cuda()
    b = torch.tensor(b0, dtype=torch.float32).cuda()
    _, mean, rstd, _ = gq.gq_layernorm_forward(x, w, b)
    dx, dw, db = (host(t) for t in gq.gq_layernorm_backward(g, w, rstd, x=x, mean=mean))

    def loss(a, ww, bb):
        return (ref.layernorm(a, ww, bb, 1e-5)[0] * gv).sum()
    wv, bv = host(w), host(b)
    for arr, grad, at in ((xv, dx, 0), (wv, dw, 1), (bv, db, 2)):
        for i in r.choice(arr.size, 12, replace=False):
            args = [xv.copy(), wv.copy(), bv.copy()]
            args[at].reshape(-1)[i] += h
            hi = loss(*args)
            args[at].reshape(-1)[i] -= 2 * h
            want = (hi - loss(*args)) / (2 * h)
            # truncation h^2 and cancellation 1e-16 / h of a loss of order 100, plus fp32
            assert abs(grad.reshape(-1)[i] - want) < 1e-4


def test_layernorm_degenerate_rows(gq, torch):
    """Constant rows (variance 0), a row with a NaN, huge and tiny rows."""
    x = np.ones((6, 200), dtype=np.float32)
    x[1] = 0.0
    x[2, 7] = np.nan
    x[3] = np.linspace(-1, 1, 200) * 1e15
    x[4] = np.linspace(-1, 1, 200) * 1e-15
    x[5] = np.linspace(-1, 1, 200)
    t, xv = tensor(torch, x, "f32")
    y, mean, rstd, act = gq.gq_layernorm_forward(t)
    wy, _, wr, hat = ref.layernorm(xv, 1.0, 0.0, 1e-5)
    near(host(y), wy, 1e-4 * (1 + np.abs(wy)), "f32")
    v = host(gq.gq_act_dequantize(act, out_dtype=torch.float32))
    assert np.isnan(v[2]).all() and not np.isnan(np.delete(v, 2, axis=0)).any()
    dx, dw, db = gq.gq_layernorm_backward(torch.ones_like(t), None, rstd, act=act)
    assert np.isnan(host(dx)[2]).all() and np.isfinite(np.delete(host(dx), 2, axis=0)).all()
    assert np.isnan(host(dw)).all() and np.array_equal(host(db), np.full(200, 6.0))


# ---- GELU ----------------------------------------------------------------------------------

def gelu_tol(u, dtype):
    # k operations on terms of size |u| and 1, a polynomial, and an exponential whose argument's
    # rounding counts as u^2 / 2 units
    poly = 5e-6 if dtype == "bf16" else 1.5e-7
    return 16 * U + poly, 4 * U * (1 + u * u)


@pytest.mark.parametrize("form", ["none", "tanh"])
@pytest.mark.parametrize("extra", [0, 3, 8])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gelu(gq, torch, rows, cols, dtype, extra, form):
    u, uv = tensor(torch, inputs(rows, cols, rows + cols, 1.5), dtype, extra)
    dh, dhv = tensor(torch, inputs(rows, cols, rows + 2 * cols, 1e-2), dtype, extra)
    h, act = gq.gq_gelu_forward(u, approximate=form, seed=5, step=6)
    rel, ex = gelu_tol(uv, dtype)
    want = ref.gelu(uv, form)[0]
    near(host(h), want, np.abs(uv) * (rel + ex * 0.2), dtype)
    wc, we = ref.quantise(uv, 5, 6)
    codes, exps = act.codes.cpu().numpy(), act.exps.cpu().numpy()
    assert np.array_equal(codes, wc) and np.array_equal(exps[:, :we.shape[1]], we)
    v = ref.values(wc, we, cols)
    wh, slope = ref.gelu(v, form)
    rel, ex = gelu_tol(v, dtype)
    du, h2 = gq.gq_gelu_backward(dh, act, approximate=form, need_output=True)
    near(host(h2), wh, np.abs(v) * (rel + ex * 0.2), dtype)
    near(host(du), dhv * slope, np.abs(dhv) * (1 + np.abs(v)) * (rel + ex), dtype)
    assert torch.equal(du, gq.gq_gelu_backward(dh, act, approximate=form))
    h3, none = gq.gq_gelu_forward(u, approximate=form, checkpoint=False)
    assert none is None and torch.equal(h, h3)


@pytest.mark.parametrize("form", ["none", "tanh"])
def test_gelu_special_values(gq, torch, form):
    u = np.zeros((2, 64), dtype=np.float32)
    u[0, :8] = [0.0, 1e30, -1e30, 30.0, -30.0, 1e-30, 5.0, -5.0]
    u[1, 0] = np.nan
    t, uv = tensor(torch, u, "f32")
    h, _ = gq.gq_gelu_forward(t, approximate=form)
    want = ref.gelu(uv, form)[0]
    rel, ex = gelu_tol(np.clip(uv, -40, 40), "f32")
    near(host(h), want, np.abs(np.clip(uv, -40, 40)) * (rel + ex * 0.2) + U * np.abs(want), "f32")
    c = np.array([[30.0, -30.0, 0.0, 127.0] * 8], dtype=np.float32)
    act = gq.gq_act_quantize(tensor(torch, c, "f32")[0])
    du = host(gq.gq_gelu_backward(torch.ones((1, 32), device="cuda"), act, approximate=form))
    assert np.allclose(du, ref.gelu(c.astype(np.float64), form)[1], atol=1e-6)


@pytest.mark.parametrize("form", ["none", "tanh"])
def test_gelu_gradient_against_differences(gq, torch, form):
    """The derivative at the checkpoint's own values against central differences."""
    x, _ = tensor(torch, np.linspace(-6, 6, 256).reshape(2, 128), "f32")
    act = gq.gq_act_quantize(x)
    v = host(gq.gq_act_dequantize(act, out_dtype=torch.float32))
    du = host(gq.gq_gelu_backward(torch.ones_like(x), act, approximate=form))
    d = 1e-5
    want = (ref.gelu(v + d, form)[0] - ref.gelu(v - d, form)[0]) / (2 * d)
    assert np.abs(du - want).max() < 1e-5


# ---- weight gradient -----------------------------------------------------------------------

WSHAPES = [(1, 1, 1), (1, 8, 32), (3, 33, 7), (63, 64, 64), (64, 128, 128), (65, 129, 130),
           (130, 100, 300), (200, 257, 255), (384, 256, 768), (1000, 640, 500), (2049, 264, 264)]


@pytest.mark.parametrize("affine_part", [False, True])
@pytest.mark.parametrize("extra", [0, 3, 8])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,outs,cols", WSHAPES)
def test_linear_wgrad(gq, torch, rows, outs, cols, dtype, out, extra, affine_part):
    x, _ = tensor(torch, inputs(rows, cols, rows + outs), dtype)
    dy, dyv = tensor(torch, inputs(rows, outs, rows + cols, 1e-2), dtype, extra)
    act = gq.gq_act_quantize(x)
    v = ref.values(act.codes.cpu().numpy(), act.exps.cpu().numpy(), cols)
    r = np.random.default_rng(1)
    scale = shift = None
    sv, hv = np.ones(cols), np.zeros(cols)
    if affine_part:
        scale, shift = (torch.tensor(a, dtype=torch.float32).cuda()
                        for a in (1 + 0.3 * r.standard_normal(cols), r.standard_normal(cols)))
        sv, hv = host(scale), host(shift)
    dw, db = gq.gq_linear_wgrad(dy, act, scale=scale, shift=shift, out_dtype=types(torch, out))
    wb = dyv.sum(axis=0)
    steps = 3 * rows if dtype == "f32" else rows
    mag = np.abs(dyv).T @ np.abs(v)
    bias = np.abs(dyv).sum(axis=0)
    tolb = (rows + 40) * U * bias
    tol = ((steps / 16 + 32) * 2.0 ** -22 + 4 * U) * mag * np.abs(sv) + \
        np.outer(tolb + 4 * U * bias, np.abs(hv))
    near(host(dw), (dyv.T @ v) * sv + np.outer(wb, hv), tol, out)
    near(host(db), wb, tolb, "f32")
    dw2, none = gq.gq_linear_wgrad(dy, act, scale=scale, shift=shift, need_bias=False,
                                   out_dtype=types(torch, out))
    assert none is None and torch.equal(dw, dw2)


@pytest.mark.parametrize("rows,outs,cols", [(4096, 1024, 768), (8192, 512, 2048), (20000, 300, 520)])
def test_linear_wgrad_large_tiles(gq, torch, rows, outs, cols):
    """Sizes that take the large tiles and share them between blocks, against a 64-bit product."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    dy = (torch.randn((rows, outs), generator=g, device="cuda") * 1e-2).bfloat16()
    act = gq.gq_act_quantize(x)
    v = gq.gq_act_dequantize(act, out_dtype=torch.float32).double()
    dw, db = gq.gq_linear_wgrad(dy, act)
    want = dy.double().t() @ v
    mag = dy.double().abs().t() @ v.abs()
    assert ((dw.double() - want).abs() <= (rows / 16 + 32) * 2.0 ** -22 * mag).all()
    assert ((db.double() - dy.double().sum(0)).abs() <= (rows + 40) * U * dy.double().abs().sum(0)).all()
    again, _ = gq.gq_linear_wgrad(dy, act)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("rows,outs,cols,dtype,out,affine_part", [
    (4096, 1024, 4096, "bf16", "f32", True), (3001, 1030, 2050, "bf16", "bf16", True),
    (16384, 520, 777, "bf16", "f32", False), (2500, 2048, 1500, "f32", "f32", True),
    (20000, 700, 300, "f32", "bf16", False), (7000, 600, 4096, "bf16", "f32", False)])
def test_linear_wgrad_pairs(gq, torch, rows, outs, cols, dtype, out, affine_part):
    """Sizes for pairs of blocks (512 x 256 tiles): several chains, shares that cross tiles, last tiles
    of fewer outs and columns, three parts of an fp32 gradient; against a 64-bit product."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    dy = (torch.randn((rows, outs), generator=g, device="cuda") * 1e-2).to(types(torch, dtype))
    act = gq.gq_act_quantize(x)
    v = gq.gq_act_dequantize(act, out_dtype=torch.float32).double()
    scale = shift = None
    s64 = torch.ones(cols, device="cuda", dtype=torch.float64)
    h64 = torch.zeros_like(s64)
    if affine_part:
        scale, shift = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda"),
                        torch.randn(cols, generator=g, device="cuda"))
        s64, h64 = scale.double(), shift.double()
    dw, db = gq.gq_linear_wgrad(dy, act, scale=scale, shift=shift, out_dtype=types(torch, out))
    d = dy.double()
    want = (d.t() @ v) * s64 + torch.outer(d.sum(0), h64)
    steps = 3 * rows if dtype == "f32" else rows
    bias = d.abs().sum(0)
    tolb = (rows + 40) * U * bias
    tol = ((steps / 16 + 32) * 2.0 ** -22 + 4 * U) * (d.abs().t() @ v.abs()) * s64.abs() + \
        torch.outer(tolb + 4 * U * bias, h64.abs()) + \
        (2.0 ** -8 if out == "bf16" else U) * want.abs()
    assert ((dw.double() - want).abs() <= tol).all()
    assert ((db.double() - d.sum(0)).abs() <= tolb).all()
    again, _ = gq.gq_linear_wgrad(dy, act, scale=scale, shift=shift, out_dtype=types(torch, out))
    assert torch.equal(dw, again)


@pytest.mark.parametrize("rows,outs,cols,dtype", [
    (1, 100, 26000, "bf16"), (3, 5, 30000, "f32"), (70, 100, 26000, "bf16"), (130, 24000, 130, "f32"),
    (40, 2100, 9000, "bf16"), (700, 2600, 1300, "f32")])
def test_linear_wgrad_many_tiles(gq, torch, rows, outs, cols, dtype):
    """More tiles than blocks, of few steps: whole tiles to each block, then shares of the rest."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    dy = (torch.randn((rows, outs), generator=g, device="cuda") * 1e-2).to(types(torch, dtype))
    shift = torch.randn(cols, generator=g, device="cuda")
    one = torch.ones_like(shift)
    act = gq.gq_act_quantize(x)
    v = gq.gq_act_dequantize(act, out_dtype=torch.float32).double()
    d = dy.double()
    dw, db = gq.gq_linear_wgrad(dy, act, scale=one, shift=shift)
    want = d.t() @ v + torch.outer(d.sum(0), shift.double())
    bias = d.abs().sum(0)
    tolb = (rows + 40) * U * bias
    steps = 3 * rows if dtype == "f32" else rows
    tol = ((steps / 16 + 32) * 2.0 ** -22 + 4 * U) * (d.abs().t() @ v.abs()) + \
        torch.outer(tolb + 4 * U * bias, shift.double().abs()) + U * want.abs()
    assert ((dw.double() - want).abs() <= tol).all()
    assert ((db.double() - d.sum(0)).abs() <= tolb).all()


def test_linear_wgrad_special_values(gq, torch):
    """A NaN block of the checkpoint reaches its columns only; an infinite gradient its row only."""
    x = np.random.default_rng(0).standard_normal((70, 96)).astype(np.float32)
    x[5, 40] = np.inf
    for dtype in DT:
        t, _ = tensor(torch, x, "f32")
        d = np.random.default_rng(1).standard_normal((70, 40)).astype(np.float32)
        d[9, 3] = np.inf
        dy, _ = tensor(torch, d, dtype)
        dw, db = gq.gq_linear_wgrad(dy, gq.gq_act_quantize(t))
        w = host(dw)
        assert np.isnan(w[:, 32:64]).all()
        others = np.delete(np.delete(w, np.s_[32:64], axis=1), 3, axis=0)
        assert np.isfinite(others).all()
        assert not np.isfinite(w[3]).any()
        assert np.isinf(host(db)[3]) and np.isfinite(np.delete(host(db), 3)).all()


# ---- large offsets, guard bands --------------------------------------------------------------

def test_offsets_past_32_bits(gq, torch):
    """2.4e9 elements (4.8 GB of bf16): the last rows equal a call of their own on the same rows."""
    rows, cols, tail = 590_000, 4096, 64
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[:tail].normal_()
    x[tail:-tail].zero_()
    x[-tail:].normal_()
    last = x[-tail:].clone()
    act = gq.gq_act_quantize(x)
    part = gq.gq_act_quantize(last)
    assert torch.equal(act.codes[-tail:], part.codes)
    v = gq.gq_act_dequantize(act)
    assert torch.equal(v[-tail:], gq.gq_act_dequantize(part))
    del v
    y, mean, rstd, ln = gq.gq_layernorm_forward(x)
    py, _, prstd, pln = gq.gq_layernorm_forward(last)
    assert torch.equal(y[-tail:], py) and torch.equal(rstd[-tail:], prstd)
    assert torch.equal(ln.codes[-tail:], pln.codes)
    del y, act
    dx, dw, db = gq.gq_layernorm_backward(x, None, rstd, act=ln)
    pdx, _, _ = gq.gq_layernorm_backward(last, None, prstd, act=pln)
    assert torch.equal(dx[-tail:], pdx)
    want = x[:tail].double().sum(0) + last.double().sum(0)
    assert torch.allclose(db.double(), want, atol=1e-3)
    del dx
    du = gq.gq_gelu_backward(x, ln)
    assert torch.equal(du[-tail:], gq.gq_gelu_backward(last, pln))


@pytest.mark.parametrize("rows,cols", [(3, 33), (5, 100), (40, 1000), (7, 1024), (320, 520), (2, 8200)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_guard_bands(gq, torch, rows, cols, dtype):
    """Through the C interface, with rows of outputs further apart than their length: nothing outside
    the outputs' own elements is written."""
    L = gq.lib()
    t = torch.float32 if dtype == 0 else torch.bfloat16
    gap, mark = 24, 123.0

    def banded(n, m):
        full = torch.full((n + 2, m + gap), mark, dtype=t, device="cuda")
        return full, full[1:-1, :m], m + gap

    def intact(full, m):
        inner = full[1:-1]
        return bool((full[0] == mark).all() and (full[-1] == mark).all() and (inner[:, m:] == mark).all())

    def banded_bytes(n, m):
        full = torch.full((n * m + 512,), 77, dtype=torch.uint8, device="cuda")
        return full, full[256:256 + n * m]

    st = torch.cuda.current_stream().cuda_stream
    pitch, epitch = gq.gq_code_pitch(cols), gq.gq_act_exp_pitch(cols)
    x = torch.randn((rows, cols), device="cuda").to(t)
    cf, c = banded_bytes(rows, pitch)
    ef, e = banded_bytes(rows, epitch)
    yf, y, ldy = banded(rows, cols)
    stats = torch.full((4 * rows,), mark, device="cuda")
    for rounding in (0, 1):
        assert L.gq_layernorm_forward(x.data_ptr(), dtype, rows, cols, cols, None, None, 0, 1e-5,
                                      y.data_ptr(), ldy, stats[rows:].data_ptr(),
                                      stats[2 * rows:].data_ptr(), rounding, 1, 1, c.data_ptr(),
                                      e.data_ptr(), st) == 0
        assert L.gq_act_quantize(x.data_ptr(), dtype, rows, cols, cols, rounding, 1, 1, c.data_ptr(),
                                 e.data_ptr(), st) == 0
    assert intact(yf, cols)
    assert (stats[:rows] == mark).all() and (stats[3 * rows:] == mark).all()
    yf, y, ldy = banded(rows, cols)
    assert L.gq_gelu_forward(x.data_ptr(), dtype, rows, cols, cols, 0, y.data_ptr(), ldy, 0, 0, 0,
                             c.data_ptr(), e.data_ptr(), st) == 0
    assert intact(yf, cols)
    for full in (cf, ef):
        assert (full[:256] == 77).all() and (full[-256:] == 77).all()
    of, o, ldo = banded(rows, cols)
    assert L.gq_act_dequantize(c.data_ptr(), e.data_ptr(), rows, cols, o.data_ptr(), dtype, ldo, st) == 0
    assert intact(of, cols)
    of, o, ldo = banded(rows, cols)
    hf, h, ldh = banded(rows, cols)
    assert L.gq_gelu_backward(x.data_ptr(), dtype, rows, cols, cols, c.data_ptr(), e.data_ptr(), 1,
                              o.data_ptr(), ldo, h.data_ptr(), ldh, st) == 0
    assert intact(of, cols) and intact(hf, cols)
    rstd = torch.ones(rows, device="cuda")
    n = L.gq_layernorm_workspace_bytes(rows, cols)
    wf, w = banded_bytes(1, n)
    of, o, ldo = banded(rows, cols)
    dw = torch.full((3, cols), mark, device="cuda")
    assert L.gq_layernorm_backward(x.data_ptr(), dtype, rows, cols, cols, None, 0, rstd.data_ptr(),
                                   c.data_ptr(), e.data_ptr(), None, 0, None, o.data_ptr(), ldo,
                                   dw[1].data_ptr(), None, 0, w.data_ptr(), n, st) == 0
    assert intact(of, cols) and (dw[0] == mark).all() and (dw[2] == mark).all()
    assert (wf[:256] == 77).all() and (wf[-256:] == 77).all()
    outs = 70
    dy = torch.randn((rows, outs), device="cuda").to(t)
    n = L.gq_linear_wgrad_workspace_bytes(dy.data_ptr(), dtype, rows, outs, outs, cols)
    wf, w = banded_bytes(1, n)
    of, o, ldo = banded(outs, cols)
    db = torch.full((3, outs), mark, device="cuda")
    assert L.gq_linear_wgrad(dy.data_ptr(), dtype, rows, outs, outs, c.data_ptr(), e.data_ptr(), cols,
                             None, None, o.data_ptr(), dtype, ldo, db[1].data_ptr(), w.data_ptr(), n,
                             st) == 0
    assert intact(of, cols) and (db[0] == mark).all() and (db[2] == mark).all()
    assert (wf[:256] == 77).all() and (wf[-256:] == 77).all()


def test_graph_capture(gq, torch):
    """A captured training step over the operators replays to the same bits."""
    x = torch.randn((256, 512), device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((256, 384), device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(512, device="cuda"), torch.zeros(512, device="cuda")

    def step():
        y, _, rstd, act = gq.gq_layernorm_forward(x, w, b, seed=1, step=2)
        dw, db = gq.gq_linear_wgrad(dy, act, scale=w, shift=b)
        h, ga = gq.gq_gelu_forward(y)
        return [y, dw, db, h, *gq.gq_layernorm_backward(gq.gq_gelu_backward(h, ga), w, rstd, act=act)]
    want = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a, c)


# ---- streams, empty inputs, refusals -------------------------------------------------------

def test_rows_zero(gq, torch):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.empty((0, 64), dtype=dtype, device="cuda")
        act = gq.gq_act_quantize(x)
        assert gq.gq_act_dequantize(act).shape == (0, 64)
        y, mean, rstd, act = gq.gq_layernorm_forward(x)
        assert y.shape == (0, 64) and mean.shape == (0,)
        dx, dw, db = gq.gq_layernorm_backward(x, None, rstd, act=act)
        assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == (64,)
        h, act = gq.gq_gelu_forward(x)
        assert gq.gq_gelu_backward(x, act).shape == (0, 64)
        dw, db = gq.gq_linear_wgrad(torch.empty((0, 40), dtype=dtype, device="cuda"), act)
        assert dw.shape == (40, 64) and not dw.any() and not db.any()


def test_leading_dimensions(gq, torch):
    x = torch.randn((2, 3, 96), device="cuda")
    y, mean, rstd, act = gq.gq_layernorm_forward(x)
    assert y.shape == x.shape and mean.shape == (6,)
    assert gq.gq_act_dequantize(act).shape == x.shape
    dx, _, _ = gq.gq_layernorm_backward(x, None, rstd, act=act)
    assert dx.shape == x.shape


def test_other_stream(gq, torch):
    """A call on a stream of its own, on inputs made on the default stream."""
    x = torch.randn((512, 640), device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((512, 256), device="cuda", dtype=torch.bfloat16)
    want = gq.gq_linear_wgrad(dy, gq.gq_act_quantize(x))
    wl = gq.gq_layernorm_forward(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    act = gq.gq_act_quantize(x, stream=s)
    got = gq.gq_linear_wgrad(dy, act, stream=s)
    gl = gq.gq_layernorm_forward(x, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(gl[0], wl[0]) and torch.equal(gl[3].codes, wl[3].codes)


def test_refusals(gq, torch):
    x = torch.randn((8, 64), device="cuda")
    act = gq.gq_act_quantize(x)
    rstd = torch.ones(8, device="cuda")
    for bad, err in ((x.double(), TypeError), (x.t(), ValueError), (x.cpu(), ValueError),
                     (x[0], ValueError), (x[:1].expand(8, 64), ValueError),
                     (x.reshape(2, 4, 64).transpose(0, 1), ValueError)):
        with pytest.raises(err):
            gq.gq_act_quantize(bad)
        with pytest.raises(err):
            gq.gq_gelu_forward(bad)
    with pytest.raises(ValueError):
        gq.gq_act_quantize(x, seed=-1)
    with pytest.raises(ValueError):
        gq.gq_act_quantize(x, seed=1, step=1 << 64)
    with pytest.raises(ValueError):
        gq.gq_gelu_forward(x, approximate="exact")
    with pytest.raises(ValueError):
        gq.gq_gelu_backward(x[:, :32].contiguous(), act)
    with pytest.raises(TypeError):
        gq.gq_gelu_backward(x, act.codes)
    with pytest.raises(ValueError):
        gq.gq_layernorm_forward(x, eps=-1.0)
    with pytest.raises(ValueError):
        gq.gq_layernorm_forward(x, torch.ones(32, device="cuda"))
    with pytest.raises(TypeError):
        gq.gq_layernorm_forward(x, torch.ones(64, device="cuda"),
                                torch.ones(64, device="cuda", dtype=torch.bfloat16))
    for kw in (dict(), dict(act=act, x=x, mean=rstd), dict(x=x), dict(act=act, mean=rstd)):
        with pytest.raises(ValueError):
            gq.gq_layernorm_backward(x, None, rstd, **kw)
    with pytest.raises(ValueError):
        gq.gq_layernorm_backward(x, None, rstd[:4], act=act)
    with pytest.raises(gq.GQError) as e:
        gq.gq_layernorm_backward(x, None, rstd, act=act, ws=torch.empty(8, device="cuda"))
    assert e.value.status == 7
    with pytest.raises(gq.GQError) as e:
        gq.gq_linear_wgrad(x, act, ws=torch.empty(64, device="cuda"))
    assert e.value.status == 7
    with pytest.raises(ValueError):
        gq.gq_linear_wgrad(x[:4], act)
    with pytest.raises(TypeError):
        gq.gq_linear_wgrad(x, act, scale=torch.ones(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gq.Act8(act.codes, act.exps, 65)
    with pytest.raises(TypeError):
        gq.Act8(act.codes.view(torch.uint8), act.exps, 64)
