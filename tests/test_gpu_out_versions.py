"""Outputs that a program gives count as changed in place: a backward pass that saved them before refuses to run."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind", ["fp8", "act"])
def test_values_in_an_output(kind):
    gq = gq_module()
    x = torch.randn((40, 96), device="cuda")
    out = torch.ones((40, 96), device="cuda")
    w = torch.randn((40, 96), device="cuda", requires_grad=True)
    loss = (w * out).sum()
    if kind == "fp8":
        gq.gq_fp8_dequantize(gq.gq_fp8_quantize(x), out=out)
    else:
        gq.gq_act_dequantize(gq.gq_act_quantize(x), out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # which count no versions
        v = torch.empty((40, 96), device="cuda")
        gq.gq_fp8_dequantize(gq.gq_fp8_quantize(x), out=v)
        gq.gq_act_dequantize(gq.gq_act_quantize(x), out=v)
