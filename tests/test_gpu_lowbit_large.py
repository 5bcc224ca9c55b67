"""8-bit floating point and AdamW on more than 2^31 elements: offsets need 64 bits.  What lies behind 2^31 is
compared bit for bit with the same rows, or elements, in a call of their own."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROWS, COLS = 600_000, 4096  # 2.46e9 elements


@pytest.fixture(scope="module")
def gq():
    return gq_module()


def test_quantise_and_back(gq):
    x = torch.empty((ROWS, COLS), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[:1000].normal_(generator=g)
    x[1000:-1000] = 1.0
    x[-1000:].normal_(generator=g)
    tail = ROWS - 1000 // 128 * 128 - ROWS % 128  # begins with a tile
    for tiles in (False, True):
        f = gq.gq_fp8_quantize(x, tiles=tiles)
        part = gq.gq_fp8_quantize(x[tail:], tiles=tiles)
        assert tail % 128 == 0 and torch.equal(f.codes[tail:].view(torch.uint8), part.codes.view(torch.uint8))
        assert torch.equal(f.blocks[tail:], part.blocks)
        back = gq.gq_fp8_dequantize(f)
        assert torch.equal(back[tail:], gq.gq_fp8_dequantize(part))
        assert torch.equal(back[5000], x[5000])
        del f, back


def test_products(gq):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((ROWS, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    w = gq.gq_fp8_quantize(torch.randn((COLS, 128), generator=g, device="cuda"), tiles=True)
    for out in (torch.bfloat16, torch.float32):
        y = gq.gq_fp8_linear(x, w, out_dtype=out)
        for a in (0, ROWS // 2 // 256 * 256, ROWS // 256 * 256 - 512):
            b = min(a + 700, ROWS)
            assert torch.equal(y[a:b], gq.gq_fp8_linear(x[a:b], w, out_dtype=out))
        del y
    # a weight and a matrix of more than 2^31 codes, summed over their long side
    dy = torch.randn((40, ROWS), generator=g, device="cuda", dtype=torch.bfloat16)
    big = gq.gq_fp8_quantize(torch.ones((ROWS, COLS), device="cuda", dtype=torch.bfloat16), tiles=True)
    got = gq.gq_fp8_linear_dgrad(dy, big, out_dtype=torch.float32)
    v = gq.gq_fp8_dequantize(gq.gq_fp8_quantize(dy), out_dtype=torch.float32).double()
    want = v.sum(1, keepdim=True)
    tol = (ROWS / 32 + 32) * 2.0 ** -22 * v.abs().sum(1, keepdim=True)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("eight", [False, True])
def test_step(gq, eight):
    n, tail = (1 << 31) + 100_003, 1 << 31
    g = torch.Generator(device="cuda").manual_seed(3)
    p = torch.zeros(n, device="cuda")
    d = torch.empty(n, device="cuda", dtype=torch.bfloat16)
    d.normal_(generator=g)
    p[tail:].normal_(generator=g)
    state = gq.gq_adamw_state(n) if eight else tuple(torch.zeros(n, device="cuda") for _ in range(2))
    q, e = p[tail:].clone(), d[tail:].clone()
    other = gq.gq_adamw_state(n - tail) if eight else tuple(torch.zeros(n - tail, device="cuda") for _ in range(2))
    norm = gq.gq_tensors_norm([d])
    want = sum(c.double().square().sum() for c in d.split(1 << 28)).sqrt()
    assert abs(norm.double() - want) <= 80 * 2.0 ** -24 * want
    for step in (1, 2):
        gq.gq_adamw_step([p], [d], [state], step, norm=norm, max_norm=1e4)
        gq.gq_adamw_step([q], [e], [other], step, norm=norm, max_norm=1e4)
    assert torch.equal(p[tail:], q)
    if eight:
        for a, b in zip(state, other):
            assert torch.equal(a[-b.shape[0]:], b)
        m, r = gq.gq_adamw_values([state])
        m2, r2 = gq.gq_adamw_values([other])
        assert torch.equal(m[0][tail:], m2[0]) and torch.equal(r[0][tail:], r2[0])
    else:
        assert all(torch.equal(a[tail:], b) for a, b in zip(state, other))
