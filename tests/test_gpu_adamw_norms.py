"""The norm that the optimizer clips by, over gradients of both types."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("a,b", [(1e18, 1e18), (1e18, 1.0), (3.0, 4.0), (0.0, 2.0), (1e-18, 1e-18)])
@pytest.mark.parametrize("dtypes", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_norm_of_both_types(a, b, dtypes):
    """Two norms joined: within 82 units of fp32 (80 a norm, 2 of the join) of the root of the sum of their squares,
    also where those are no fp32 numbers."""
    gq_module()
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    params = [torch.nn.Parameter(torch.zeros(1024, device="cuda", dtype=t)) for t in dtypes]
    for p, v in zip(params, (a, b)):
        p.grad = torch.full_like(p, v)
    opt = AdamW(params, max_norm=1.0, weight_decay=0.0, lr=1e-3, states="f32")
    want = sum(p.grad.double().square().sum() for p in params).sqrt()
    got = opt._norm([p.grad for p in params])
    assert got.numel() == 1 and got.dtype == torch.float32
    assert abs(got.double() - want) <= 82 * 2.0 ** -24 * want
    opt.step()
    clip = min(1.0, 1.0 / (float(want) + 1e-6))
    for p in params:
        m = 0.1 * p.grad.double() * clip
        assert ((opt.state[p]["m"].double() - m).abs() <= 92 * 2.0 ** -24 * m.abs()).all()


def test_other_types_are_refused_by_name():
    gq_module()
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    p = torch.nn.Parameter(torch.zeros(4, device="cuda", dtype=torch.float16))
    p.grad = torch.ones_like(p)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        AdamW([p], max_norm=1.0).step()
    q = torch.nn.Parameter(torch.zeros(4, device="cuda"))
    q.grad = torch.ones_like(q)
    opt = AdamW([q, p], max_norm=1.0)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        opt.step()
    assert not q.any()
