"""How exact the sums of the products in 8-bit floating point are, and where weights of more than 2^31 codes are
read."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gq():
    return gq_module()


@pytest.mark.parametrize("depth", [128, 1024, 4096, 8192])
@pytest.mark.parametrize("rows", [100, 2560])
@pytest.mark.parametrize("gradient", [False, True])
def test_relative_error(gq, rows, depth, gradient):
    """Normal numbers, fp32 results, calls of both forms: within twice the part of the result's norm that is stated
    for one chain of 8,192, 4.9e-7, in proportion to the depth, and a rounding.

    In proportion: a chain adds 32 products at a time and cuts the sum each time, by a part c of it in the mean and
    towards zero, so that its error is c times the sum of its n = depth / 32 partial sums S_j.  These are a random
    walk: the sum of them has n^3 / 3 times the variance of a step, the last one n times, so the relative
    error is c n / sqrt(3).  Parts of a sum, added in the end, have shorter chains."""
    g = torch.Generator(device="cuda").manual_seed(depth + rows)
    x = gq.gq_fp8_quantize(torch.randn((rows, depth), generator=g, device="cuda"))
    shape = (depth, 1280) if gradient else (1280, depth)
    w = gq.gq_fp8_quantize(torch.randn(shape, generator=g, device="cuda"), tiles=True)
    xv, wv = (gq.gq_fp8_dequantize(f, out_dtype=torch.float32).double() for f in (x, w))
    want = xv @ (wv if gradient else wv.t())
    got = (gq.gq_fp8_linear_dgrad if gradient else gq.gq_fp8_linear)(x, w, out_dtype=torch.float32)
    off = float((got.double() - want).norm() / want.norm())
    print("rows %d depth %d gradient %d: %.2e" % (rows, depth, gradient, off))
    assert off <= 2 * 4.9e-7 * depth / 8192 + 2.0 ** -24


def test_codes_behind_2_31_by_value(gq):
    """Small integers that e4m3 holds, other ones at every place, so that sums are exact: rows on both sides of
    2^31 bytes are those that are asked for."""
    outs, cols = 600_000, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty((outs, cols), dtype=torch.bfloat16, device="cuda")
    for part in w.split(1 << 16):
        part.copy_(torch.randint(-8, 9, part.shape, generator=g, device="cuda", dtype=torch.int8))
    f = gq.gq_fp8_quantize(w, tiles=True)
    edge = (1 << 31) // cols
    some = [0, 1, 5000, edge - 129, edge - 2, edge - 1, edge, edge + 1, edge + 128, outs - 130, outs - 1]
    for rows in (3, 300):
        dy = torch.zeros((rows, outs), dtype=torch.bfloat16, device="cuda")
        v = torch.randint(-8, 9, (rows, len(some)), generator=g, device="cuda").float()
        dy[:, some] = v.bfloat16()
        got = gq.gq_fp8_linear_dgrad(dy, f, out_dtype=torch.float32)
        assert torch.equal(got.double(), v.double() @ w[some].double())
        del dy, got
        x = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").bfloat16()
        y = gq.gq_fp8_linear(x, f, out_dtype=torch.float32)
        at = 0
        for part in w.split(1 << 16):
            # sums of integers below 2^24: exact in fp32 in any order
            want = x.float() @ part.float().t()
            assert torch.equal(y[:, at:at + part.shape[0]], want)
            at += part.shape[0]
        del y
