"""What blocks with products in 8-bit floating point keep for the backward pass: weights in 8 bits only where an input's
gradient will be computed from them."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("frozen,of_x,kept", [((), True, 2), ((), False, 2), (("norm_weight", "norm_bias"), False, 1),
                                              (("norm_weight", "norm_bias", "w1"), False, 1),
                                              (("norm_weight", "norm_bias", "w1", "b1"), False, 1),
                                              (("norm_weight", "norm_bias", "w1", "b1", "w2"), False, 0),
                                              (("norm_weight", "norm_bias", "w1", "b1", "w2"), True, 2)])
def test_weights_in_8_bits_that_are_kept(frozen, of_x, kept):
    gq_module()
    from allreduce_compatible_gradient_gb300.act8_layers import MlpBlock8
    torch.manual_seed(1)
    block = MlpBlock8(96, 200, device="cuda", seed=1, products="e4m3")
    for name, p in block.named_parameters():
        p.requires_grad_(name not in frozen)
    x = torch.randn((33, 96), device="cuda", requires_grad=of_x)
    found = []

    def pack(t):
        if t.dtype == torch.uint8 and t.dim() == 1:  # (checkpoints are matrices)
            found.append(t.numel())
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        out = block(x)
    assert len(found) == kept, found
    out.sum().backward()
    for name, p in block.named_parameters():
        assert (p.grad is None) == (name in frozen)
    assert (x.grad is not None) == of_x
