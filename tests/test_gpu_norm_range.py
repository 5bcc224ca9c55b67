"""The norm of many tensors where sums of squares pass fp32's range, and where its workspace lies."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def gq():
    return gq_module()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,size", [([64], 1.7e19), ([1000], 1e19), ([40000, 7, 3], 1e18), ([1 << 22, 12345], 1e18),
                                        ([50] * 300, 9e18), ([3 << 25], 1.5e17)], ids=str)
def test_large_magnitudes(gq, dtype, sizes, size):
    """Magnitudes whose squares are fp32 numbers, and whose sum is not: the norm is the sum's root all the same."""
    g = torch.Generator(device="cuda").manual_seed(1)
    t = [((torch.rand(n, generator=g, device="cuda") * 0.5 + 0.5) * size).to(dtype) for n in sizes]
    want = torch.stack([c.double().square().sum() for x in t for c in x.split(1 << 24)]).sum().sqrt()
    got = gq.gq_tensors_norm(t)
    assert abs(got.double() - want) <= 80 * U * want
    assert torch.equal(got, gq.gq_tensors_norm(t))


def test_large_magnitudes_among_others(gq):
    """A few large ones in one tensor of many, in any place; a NaN or an infinity anywhere still leaves no number."""
    t = [torch.ones(n, device="cuda") for n in (5000, 300000, 70)]
    flat = t[1]
    for at in (0, 150001, 299999):
        flat[at:at + 40] = 1e19
        want = torch.stack([x.double().square().sum() for x in t]).sum().sqrt()
        assert abs(gq.gq_tensors_norm(t).double() - want) <= 80 * U * want
        for bad in (float("nan"), float("inf"), -float("inf")):
            for x, k in ((t[0], 7), (flat, 200000), (t[2], 69)):
                x[k] = bad
                assert not gq.gq_tensors_norm(t).isfinite().any()
                x[k] = 1.0
        flat[at:at + 40] = 1.0


def test_a_step_with_a_large_norm_is_made(gq):
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    p = torch.nn.Parameter(torch.zeros(5000, device="cuda"))
    p.grad = torch.full((5000,), 1e18, device="cuda")
    AdamW([p], lr=1e-3, max_norm=1.0, weight_decay=0.0).step()
    assert ((p + 1e-3).abs() <= 1e-6).all()


def test_small_magnitudes(gq):
    """Squares are fp32 numbers, also below the normal ones: digits go below 1.1e-19, all of them below 2.6e-23."""
    for size, off in ((1.2e-19, 80 * U), (1e-21, 2.0 ** -8), (2.5e-23, 1.0)):
        t = [torch.full((n,), size, device="cuda") for n in (1000, 33)]
        want = 1033 ** 0.5 * size
        got = gq.gq_tensors_norm(t).item()
        assert abs(got - want) <= off * want
    assert gq.gq_tensors_norm([torch.full((1000,), 2.5e-23, device="cuda")]).item() == 0.0
