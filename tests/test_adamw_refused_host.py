"""A step that is refused is not counted, on a machine without a GPU: calls are recorded in place of the native
entry point."""
import pytest

torch = pytest.importorskip("torch")


class Recorder:
    """Stands for the native module: (parameter, its step's number) of every update; bf16 parameters are refused
    while `refuse`."""

    def __init__(self):
        self.calls, self.refuse = [], False

    def adamw_step(self, params, grads, states, step, *rest):
        if self.refuse and params[0].dtype == torch.bfloat16:
            raise ValueError("refused")
        for i, p in enumerate(params):
            self.calls.append((p, int(step if rest[10] is None else step[rest[10][i]])))


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_is_not_counted(monkeypatch, capturable):
    """Two parameters of either type in a group: the call for one type has been made, the other's is refused."""
    from allreduce_compatible_gradient_gb300 import _activations
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    record = Recorder()
    monkeypatch.setattr(_activations, "_native", record)
    params = [torch.nn.Parameter(torch.zeros(4, dtype=t)) for t in (torch.float32, torch.bfloat16) * 2]
    opt = AdamW(params, capturable=capturable)
    for p in params:
        p.grad = torch.ones_like(p)
    opt.step()
    record.refuse = True
    for _ in range(2):
        with pytest.raises(ValueError):
            opt.step()
    record.refuse = False
    del record.calls[:]
    opt.step()
    got = {id(p): t for p, t in record.calls}
    assert [got[id(p)] for p in params] == [4, 2, 4, 2]
    assert [int(opt.state[p]["step"]) for p in params] == [4, 2, 4, 2]
