"""The choice of the layers' products, on a machine without a GPU: what is not a choice is refused before any
operator is called."""
import copy

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bad", ["fp8", "E4M3", None, True, ""])
def test_unknown_products_are_refused(monkeypatch, bad):
    from allreduce_compatible_gradient_gb300 import act8_layers
    called = []
    for name in ("_NormLinear", "_GeluLinear"):
        fake = type(name, (), {"apply": staticmethod(lambda x, *a: called.append(a[-1]) or x)})
        monkeypatch.setattr(act8_layers, name, fake)
    with pytest.raises(ValueError, match="products"):
        act8_layers.MlpBlock8(8, 16, products=bad)
    block = act8_layers.MlpBlock8(8, 16)
    x = torch.zeros(2, 8)
    for choice in ("bf16", "e4m3"):
        block.products = choice
        block(x)
    assert called == [False, False, True, True]
    block.products = bad
    for b in (block, copy.deepcopy(block)):
        with pytest.raises(ValueError, match="products"):
            b(x)
    assert len(called) == 4
