"""The optimizer under a graph capture without `capturable`, on a machine without a GPU: whether a capture runs is
asked of torch, which a test can answer for."""
import pytest

torch = pytest.importorskip("torch")


class Recorder:
    calls = 0

    def adamw_step(self, *args):
        self.calls += 1


def test_numbers_of_the_host_are_not_captured(monkeypatch):
    """A graph would repeat the number of its capture at every replay: refused, and nothing is counted."""
    from allreduce_compatible_gradient_gb300 import _activations
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    record = Recorder()
    monkeypatch.setattr(_activations, "_native", record)
    p = torch.nn.Parameter(torch.zeros(4))
    p.grad = torch.ones(4)
    opt = AdamW([p])
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="capturable"):
        opt.step()
    assert record.calls == 1 and int(opt.state[p]["step"]) == 1
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    opt.step()
    assert record.calls == 2 and int(opt.state[p]["step"]) == 2
