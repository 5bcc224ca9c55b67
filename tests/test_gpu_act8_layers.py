"""The layers over 8-bit checkpoints: gradients against autograd's in fp64, unbiasedness of the weight
gradient, and the training example."""
import importlib.util
import os

import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layers():
    gq_module()
    from allreduce_compatible_gradient_gb300 import act8_layers
    return act8_layers


def block_of(layers, dtype, approximate="none"):
    torch.manual_seed(3)
    block = layers.MlpBlock8(96, 200, approximate=approximate, seed=5, device="cuda")
    with torch.no_grad():
        for p in block.parameters():
            p += 0.1 * torch.randn_like(p)
    return block, torch.randn((2, 75, 96), device="cuda").to(dtype)


def exact_gradients(block, x, r):
    """Autograd's, in fp64, of sum(block(x) r)."""
    p = {k: v.detach().double().requires_grad_() for k, v in block.named_parameters()}
    x = x.detach().double().requires_grad_()
    y = torch.nn.functional.layer_norm(x, x.shape[-1:], p["norm_weight"], p["norm_bias"], block.eps)
    h = torch.nn.functional.gelu(y @ p["w1"].t() + p["b1"], approximate=block.approximate)
    out = x + h @ p["w2"].t() + p["b2"]
    g = torch.autograd.grad((out * r.double()).sum(), [x, *p.values()])
    return out, dict(zip(["x", *p], g))


@pytest.mark.parametrize("approximate", ["none", "tanh"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_near_autograd(layers, dtype, approximate):
    """A code's error is within a step, at most 1/64 of its block's largest value, about 0.6 of the step
    in the mean square when rounded at random; of the bf16 products' inputs 2^-9 each.  Sums over 150 rows
    average both out: 2 % of a gradient's norm is several times what is left."""
    block, x = block_of(layers, dtype, approximate)
    x.requires_grad_()
    r = torch.randn((2, 75, 96), device="cuda")
    out = block(x)
    got = torch.autograd.grad((out.float() * r).sum(), [x, *block.parameters()])
    want_out, want = exact_gradients(block, x, r)
    assert (out.double() - want_out).norm() < 0.01 * want_out.norm()
    for g, (name, w) in zip(got, want.items()):
        assert (g.double() - w).norm() < 0.02 * w.norm(), name


def test_weight_gradient_is_unbiased(layers):
    """Over many steps the mean of w1's gradient approaches the exact one as 1 / sqrt(steps)."""
    block, x = block_of(layers, torch.float32)
    r = torch.randn((2, 75, 96), device="cuda")
    _, want = exact_gradients(block, x, r)
    # the upstream gradient of w1 depends on the GELU checkpoint too: only the first layer's rounding
    # is averaged here, with its output's gradient held fixed
    from allreduce_compatible_gradient_gb300 import act8_layers as L
    dout = torch.randn((150, 200), device="cuda")
    rows = x.reshape(-1, 96)
    y = torch.nn.functional.layer_norm(rows.double(), (96,), block.norm_weight.double(),
                                       block.norm_bias.double(), block.eps)
    exact = dout.double().t() @ y
    total, one, n = 0, None, 100
    for step in range(n):
        w = block.w1.detach().requires_grad_()
        out = L._NormLinear.apply(rows, block.norm_weight, block.norm_bias, w, block.b1, block.eps, 9, step)
        g, = torch.autograd.grad((out * dout).sum(), [w])
        one = (g.double() - exact).norm() if one is None else one
        total = total + g.double()
    assert (total / n - exact).norm() < 2 * one / n ** 0.5


def test_training_example_learns():
    gq_module()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_mlp8.py")
    spec = importlib.util.spec_from_file_location("train_mlp8", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(workers=2, steps=12, width=64, hidden=128, tokens=256)
    assert all(v == v for v in losses) and losses[-1] < 0.8 * losses[0]
