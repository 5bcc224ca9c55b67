"""8-bit floating point and the products of linear layers on it, against their definitions in 64 bits.

Tolerances, with u = 2^-24 (half a unit in the last place of fp32):
- codes and exponents are exact: a product with a power of two and one rounding;
- the tensor cores add 32 products of codes (exact in fp32, scales are powers of two) at a time and may
  truncate, 2^-22 of the largest partial sum a time, and up to 8 parts of a sum and a bias are added in fp32:
  within (k / 32 + 32) 2^-22 of the sum of the magnitudes;
- the result is rounded once: 2^-8 of its magnitude in bf16, u in fp32.
"""
import pytest

import lowbit_ref as ref
from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gq():
    return gq_module()


def matrix(rows, cols, dtype, seed, extra=0, shift=0):
    """Normal numbers with columns of unequal scale, a row and a block of zeros, in rows cols + extra apart
    that begin `shift` elements into a buffer of NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(torch.randn(cols, generator=g, device="cuda"))
    if rows > 2:
        x[rows // 2] = 0.0
    if cols > 300:
        x[0, 128:256] = 0.0
    if extra == 0 and shift == 0:
        return x.to(TYPES[dtype])
    flat = torch.full((rows * (cols + extra) + shift,), float("nan"), dtype=TYPES[dtype], device="cuda")
    out = flat[shift:].view(rows, cols + extra)[:, :cols]
    out.copy_(x)
    return out


def check(f, x, tiles):
    """An Fp8's codes, exponents and padding against the definition."""
    q, e = ref.fp8(x, 128 if tiles else 1)
    rows, cols = x.shape
    codes = f.codes.float().double()
    assert codes.shape == (rows, (cols + 15) // 16 * 16)
    assert torch.equal(codes[:, :cols], q) and not codes[:, cols:].any()
    want = e.repeat_interleave(128, dim=0)[:rows] if tiles else e
    assert torch.equal(f.blocks.long(), want)
    if tiles:
        t = f.exps_t.permute(0, 3, 2, 1, 4)
        t = t.reshape(t.shape[0] * 128, -1)[:cols, :(rows + 127) // 128]
        assert torch.equal(t.long(), e.t().repeat_interleave(128, dim=0)[:cols])
    return ref.values(q, e, 128 if tiles else 1)


SIZES = [(1, 1), (1, 128), (3, 129), (5, 16), (31, 511), (128, 512), (129, 513), (200, 1000), (64, 2049),
         (257, 640), (1000, 96)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize(gq, rows, cols, dtype, tiles):
    x = matrix(rows, cols, dtype, rows + cols)
    f = gq.gq_fp8_quantize(x, tiles=tiles)
    want = check(f, x, tiles)
    assert f.shape == x.shape and f.rows == rows and f.cols == cols and f.tiles == tiles
    for out in (torch.float32, torch.bfloat16, torch.float16):
        got = gq.gq_fp8_dequantize(f, out_dtype=out)
        assert got.dtype == out and torch.equal(got, want.to(torch.float32).to(out))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("extra,shift", [(3, 0), (8, 0), (0, 1), (5, 3), (64, 8)])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_strides(gq, dtype, extra, shift, tiles):
    """Rows of any distance and alignment; nothing beside them is read into a block, outputs likewise."""
    for rows, cols in ((37, 260), (140, 1030)):
        x = matrix(rows, cols, dtype, 7, extra, shift)
        f = gq.gq_fp8_quantize(x, tiles=tiles)
        want = check(f, x, tiles)
        out = matrix(rows, cols, dtype, 8, extra, shift)
        before = out.untyped_storage()
        beside = torch.empty(0, dtype=out.dtype, device="cuda").set_(before).clone()
        gq.gq_fp8_dequantize(f, out=out)
        assert torch.equal(out, want.to(torch.float32).to(out.dtype))
        after = torch.empty(0, dtype=out.dtype, device="cuda").set_(before)
        mask = torch.ones_like(after, dtype=torch.bool)
        mask[shift:].view(rows, cols + extra)[:, :cols] = False
        assert torch.equal(after[mask].isnan(), beside[mask].isnan())


def test_quantize_special_values(gq):
    """Borders of the exponent rule, ties, subnormal magnitudes, and blocks that are not finite."""
    x = torch.zeros((12, 256), device="cuda")
    x[0, 0], x[0, 130] = 448.0, 448.0 * (1 + 2.0 ** -23)      # the largest of a step, and just above
    x[1, :8] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, -18.0, 0.4999 * 2.0 ** -9])
    x[2, 5], x[2, 200] = float("inf"), 1.0
    x[3, 5], x[3, 200] = float("nan"), -2.0
    x[4, :3] = torch.tensor([2.0 ** -149, -2.0 ** -130, 2.0 ** -127])
    x[5, :2] = torch.tensor([3.4028234e38, 1.0])
    x[6, 0] = -float("inf")
    x[7, :2] = torch.tensor([1.0, -0.0])
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        f = gq.gq_fp8_quantize(y)
        want = check(f, y, False)
        got = gq.gq_fp8_dequantize(f, out_dtype=torch.float32)
        assert torch.equal(got.isnan(), want.isnan()) and got[2, :128].isnan().all()
        assert torch.equal(got.nan_to_num(), want.to(torch.float32).nan_to_num())
        t = gq.gq_fp8_quantize(y, tiles=True)
        q, e = ref.fp8(y, 128)
        assert torch.equal(t.blocks.long(), e.expand(12, 2)) and torch.equal(t.codes.float().double(), q)


def test_no_rows(gq):
    x = torch.empty((0, 300), device="cuda", dtype=torch.bfloat16)
    f = gq.gq_fp8_quantize(x)
    assert f.rows == 0 and gq.gq_fp8_dequantize(f).shape == (0, 300)
    w = gq.gq_fp8_quantize(matrix(70, 300, "f32", 1), tiles=True)
    assert gq.gq_fp8_linear(x, w).shape == (0, 70) and gq.gq_fp8_linear(f, w).shape == (0, 70)
    d = torch.empty((2, 0, 70), device="cuda")
    assert gq.gq_fp8_linear_dgrad(d, w).shape == (2, 0, 300)


# ---- products ------------------------------------------------------------------------------

def near(got, want, total, k):
    """Within the tolerance of a product over k terms whose magnitudes add up to `total`."""
    tol = (k / 32 + 32) * 2.0 ** -22 * total + (2.0 ** -8 if got.dtype == torch.bfloat16 else U) * want.abs()
    d = (got.double() - want).abs()
    assert got.shape == want.shape and (d <= tol).all(), (d.max(), (d / tol.clamp(min=1e-300)).max())


def forward(gq, rows, cols, outs, dtype, out, tiles=True, bias=True, seed=0, extra=0, shift=0):
    x = matrix(rows, cols, dtype, seed + 1, extra, shift)
    w = matrix(outs, cols, "f32", seed + 2) * cols ** -0.5
    b = torch.randn(outs, device="cuda") if bias else None
    f = gq.gq_fp8_quantize(w, tiles=tiles)
    xv, wv = ref.values(*ref.fp8(x, 1), 1), ref.values(*ref.fp8(w, 128 if tiles else 1), 128 if tiles else 1)
    want, total = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if bias:
        want, total = want + b.double(), total + b.double().abs()
    got = gq.gq_fp8_linear(x, f, bias=b, out_dtype=TYPES[out])
    near(got, want, total, cols)
    # the same from a matrix that is in 8 bits already
    assert torch.equal(got, gq.gq_fp8_linear(gq.gq_fp8_quantize(x), f, bias=b, out_dtype=TYPES[out]))
    return got


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 4096, 512), (2, 130, 100), (5, 640, 129), (16, 512, 256), (17, 1000, 40),
            (33, 2048, 300), (64, 96, 1000), (65, 1300, 700), (100, 256, 1024), (128, 768, 768), (200, 513, 127),
            (384, 768, 768), (1021, 1001, 2050), (2000, 700, 900), (3000, 2560, 1024), (2100, 1300, 2100),
            (4000, 260, 1100), (300, 520, 12000), (9000, 2100, 700), (2500, 4096, 2304), (17000, 200, 250)]


@pytest.mark.parametrize("rows,cols,outs", PRODUCTS)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_linear(gq, rows, cols, outs, dtype, out):
    forward(gq, rows, cols, outs, dtype, out)


@pytest.mark.parametrize("rows,cols,outs", PRODUCTS)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16")])
def test_linear_dgrad(gq, rows, cols, outs, dtype, out):
    dy = matrix(rows, outs, dtype, 3)
    w = matrix(outs, cols, "f32", 4) * cols ** -0.5
    f = gq.gq_fp8_quantize(w, tiles=True)
    d, wv = ref.values(*ref.fp8(dy, 1), 1), ref.values(*ref.fp8(w, 128), 128)
    got = gq.gq_fp8_linear_dgrad(dy, f, out_dtype=TYPES[out])
    near(got, d @ wv, d.abs() @ wv.abs(), outs)
    assert torch.equal(got, gq.gq_fp8_linear_dgrad(gq.gq_fp8_quantize(dy), f, out_dtype=TYPES[out]))


@pytest.mark.parametrize("rows,cols,outs,dtype", [(16300, 2048, 1024, "bf16"), (16384, 4096, 4096, "bf16"),
                                                  (9800, 2100, 1000, "f32")])
def test_many_waves_of_tiles(gq, rows, cols, outs, dtype):
    """Long x: bit for bit the result of the same matrix put into 8 bits before, over and over with nothing waiting in
    between, and replayed from a graph; some rows against 64 bits."""
    w = matrix(outs, cols, "f32", 2)
    f = gq.gq_fp8_quantize(w, tiles=True)
    xs = [matrix(rows, cols, dtype, k) for k in range(2)]
    want = [gq.gq_fp8_linear(gq.gq_fp8_quantize(x), f, out_dtype=torch.bfloat16) for x in xs]
    some = torch.randint(0, rows, (200,), device="cuda")
    xv, wv = ref.values(*ref.fp8(xs[0][some], 1), 1), ref.values(*ref.fp8(w, 128), 128)
    near(want[0][some], xv @ wv.t(), xv.abs() @ wv.abs().t(), cols)
    for _ in range(4):
        got = [gq.gq_fp8_linear(x, f, out_dtype=torch.bfloat16) for x in xs]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    x = xs[0].clone()
    with torch.cuda.graph(graph):
        y = gq.gq_fp8_linear(x, f, out_dtype=torch.bfloat16)
        z = y.sum()
    for k in (0, 1, 0):
        x.copy_(xs[k])
        y.zero_()
        graph.replay()
        assert torch.equal(y, want[k]) and torch.equal(z, want[k].sum())


def test_linear_weights_by_rows(gq):
    """A weight with an exponent per row's block, and no bias."""
    forward(gq, 77, 1500, 333, "bf16", "bf16", tiles=False, bias=False)
    forward(gq, 500, 640, 640, "f32", "f32", tiles=False)


@pytest.mark.parametrize("extra,shift", [(3, 0), (0, 1), (8, 8)])
def test_linear_strides(gq, extra, shift):
    forward(gq, 50, 700, 200, "bf16", "bf16", extra=extra, shift=shift)
    forward(gq, 300, 260, 200, "f32", "f32", extra=extra, shift=shift)


def test_linear_leading_dimensions(gq):
    x = torch.randn((3, 5, 260), device="cuda", dtype=torch.bfloat16)
    f = gq.gq_fp8_quantize(torch.randn((70, 260), device="cuda"), tiles=True)
    y = gq.gq_fp8_linear(x, f)
    assert y.shape == (3, 5, 70) and y.dtype == torch.bfloat16
    assert torch.equal(y.view(15, 70), gq.gq_fp8_linear(x.view(15, 260), f))
    assert gq.gq_fp8_linear(gq.gq_fp8_quantize(x), f).shape == (3, 5, 70)
    assert gq.gq_fp8_linear_dgrad(y, f).shape == (3, 5, 260)


def test_linear_not_finite(gq):
    """A block that is not finite reaches the sums that it takes part in and no other: its token's in the
    forward pass, its outputs' of every token where it is the weight's."""
    x, w = torch.randn((200, 500), device="cuda"), torch.randn((300, 500), device="cuda")
    x[7, 3], x[130, 450] = float("inf"), float("nan")
    f = gq.gq_fp8_quantize(w, tiles=True)
    y = gq.gq_fp8_linear(x, f)
    bad = torch.zeros(200, dtype=torch.bool, device="cuda")
    bad[7] = bad[130] = True
    assert y[bad].isnan().all() and y[~bad].isfinite().all()
    w[140, 9] = float("nan")
    x = torch.randn((200, 500), device="cuda")
    y = gq.gq_fp8_linear(x, gq.gq_fp8_quantize(w, tiles=True))
    assert y[:, 128:256].isnan().all() and y[:, :128].isfinite().all() and y[:, 256:].isfinite().all()
    y = gq.gq_fp8_linear(x, gq.gq_fp8_quantize(w))
    assert y[:, 140].isnan().all() and y.isnan().sum() == 200


@pytest.mark.parametrize("rows", [1, 16, 40])
def test_linear_not_finite_few_tokens(gq, rows):
    x, w = torch.randn((rows, 700), device="cuda"), torch.randn((300, 700), device="cuda")
    x[rows - 1, 600] = -float("inf")
    y = gq.gq_fp8_linear(x, gq.gq_fp8_quantize(w, tiles=True))
    assert y[rows - 1].isnan().all() and y[:rows - 1].isfinite().all()


@pytest.mark.parametrize("rows,outs", [(1, 200), (9, 131), (50, 200), (300, 131), (4200, 1030), (4200, 1032)])
@pytest.mark.parametrize("ldy,shift", [(0, 0), (8, 0), (2, 0), (1, 0), (8, 8), (8, 1)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_outputs_of_any_place(gq, rows, outs, ldy, shift, out):
    """The C entry: rows of y further apart than their length and at any element; what lies between them stays."""
    cols, ld = 260, outs + ldy
    x, w = matrix(rows, cols, "bf16", 1), gq.gq_fp8_quantize(matrix(outs, cols, "f32", 2), tiles=True)
    want = gq.gq_fp8_linear(x, w, out_dtype=TYPES[out])
    f = gq.gq_fp8_quantize(x)
    for given in (None, x):
        room = torch.full((rows * ld + shift + 8,), 7.0, dtype=TYPES[out], device="cuda")
        y = room[shift:]
        codes, exps = f.codes.clone(), f.exps.clone()
        if given is not None and gq.gq_fp8_linear_workspace_bytes(rows, cols, outs) == 0:
            codes = exps = torch.empty(0)  # null: none is needed
        status = gq.lib().gq_fp8_linear(None if given is None else given.data_ptr(), gq.BF16, cols, codes.data_ptr(),
                                        exps.data_ptr(), rows, cols, w.codes.data_ptr(), w.exps.data_ptr(), outs, None,
                                        y.data_ptr(), gq.BF16 if out == "bf16" else gq.F32, ld,
                                        torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        body = y[:rows * ld].view(rows, ld)
        assert torch.equal(body[:, :outs], want)
        assert (body[:, outs:] == 7).all() and (room[:shift] == 7).all() and (room[shift + rows * ld:] == 7).all()


def test_linear_extreme_scales(gq):
    """Blocks whose scales differ by 2^60 within a sum, and sums near the ends of fp32's range."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((40, 640), generator=g, device="cuda")
    x[:, 128:256] *= 2.0 ** 60
    x[:, 256:384] *= 2.0 ** -60
    w = torch.randn((130, 640), generator=g, device="cuda") * 2.0 ** 20
    f = gq.gq_fp8_quantize(w, tiles=True)
    xv, wv = ref.values(*ref.fp8(x, 1), 1), ref.values(*ref.fp8(w, 128), 128)
    near(gq.gq_fp8_linear(x, f), xv @ wv.t(), xv.abs() @ wv.abs().t(), 640)


def test_zero_operand(gq):
    x = torch.zeros((130, 300), device="cuda")
    f = gq.gq_fp8_quantize(torch.randn((70, 300), device="cuda"), tiles=True)
    assert not gq.gq_fp8_linear(x, f).any()
    b = torch.randn(70, device="cuda")
    assert torch.equal(gq.gq_fp8_linear(x, f, bias=b), b.expand(130, 70))


def test_one_hot_rows_pick_the_weights_columns(gq):
    """Every element of the weight arrives at its place: products with the unit matrix give its values, both
    ways."""
    w = matrix(390, 650, "f32", 11)
    f = gq.gq_fp8_quantize(w, tiles=True)
    v = ref.values(*ref.fp8(w, 128), 128).float()
    assert torch.equal(gq.gq_fp8_linear(torch.eye(650, device="cuda"), f), v.t())
    assert torch.equal(gq.gq_fp8_linear_dgrad(torch.eye(390, device="cuda"), f), v)
