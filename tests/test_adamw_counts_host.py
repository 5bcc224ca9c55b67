"""Which step numbers the optimizer gives to which parameter, on a machine without a GPU: its calls are recorded
in place of the native entry point."""
import copy
import ctypes
import io

import pytest

torch = pytest.importorskip("torch")


class Recorder:
    """Stands for the native module: (parameter, its step's number) of every update."""

    def __init__(self):
        self.calls = []

    def tensors_norm(self, tensors, ws):
        return torch.ones(1)

    def adamw_step(self, params, grads, states, step, *rest):
        counted = rest[10] if len(rest) > 10 else None
        for i, p in enumerate(params):
            self.calls.append((p, int(step if counted is None else step[counted[i]])))


@pytest.fixture
def record(monkeypatch):
    from allreduce_compatible_gradient_gb300 import _activations
    recorder = Recorder()
    monkeypatch.setattr(_activations, "_native", recorder)
    return recorder


def made(n=3, groups=1, **kw):
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    params = [torch.nn.Parameter(torch.zeros(4)) for _ in range(n)]
    return params, AdamW([dict(params=params[i::groups]) for i in range(groups)], **kw)


def step(record, opt, params, which):
    """The numbers that the parameters of `which` get."""
    for i, p in enumerate(params):
        p.grad = torch.ones_like(p) if i in which else None
    del record.calls[:]
    opt.step()
    got = {id(p): t for p, t in record.calls}
    assert len(record.calls) == len(which)
    return [got[id(params[i])] for i in which]


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("groups", [1, 2])
def test_own_updates_are_counted(record, capturable, groups):
    """A parameter that joins late begins with 1, one that is left out in some steps counts its own."""
    params, opt = made(groups=groups, capturable=capturable)
    assert step(record, opt, params, [0]) == [1]
    assert step(record, opt, params, [0, 1]) == [2, 1]
    assert step(record, opt, params, [1]) == [2]
    assert step(record, opt, params, [0, 1, 2]) == [3, 3, 1]
    assert step(record, opt, params, [2]) == [2]
    assert step(record, opt, params, [0, 1, 2]) == [4, 4, 3]
    assert [int(opt.state[p]["step"]) for p in params] == [4, 4, 3]


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("how", ["file", "deep copy", "state of its own"])
def test_counts_are_kept(record, capturable, how):
    params, opt = made(groups=2, capturable=capturable)
    for which in ([0], [0, 1], [1]):
        step(record, opt, params, which)
    if how == "deep copy":
        opt = copy.deepcopy(opt)
        params = [opt.param_groups[i % 2]["params"][i // 2] for i in range(3)]
    else:
        saved = opt.state_dict()
        if how == "file":
            f = io.BytesIO()
            torch.save(saved, f)
            f.seek(0)
            saved = torch.load(f)
        others, other = made(groups=2, capturable=capturable)
        other.load_state_dict(saved)
        # the first one's counts are its own
        assert step(record, opt, params, [0, 1, 2]) == [3, 3, 1]
        params, opt = others, other
    assert step(record, opt, params, [0, 1, 2]) == [3, 3, 1]


@pytest.mark.parametrize("before,after", [(False, True), (True, False)])
def test_counts_pass_between_kinds(record, before, after):
    params, opt = made(capturable=before)
    for which in ([0], [0, 1]):
        step(record, opt, params, which)
    others, other = made(capturable=after)
    other.load_state_dict(opt.state_dict())
    assert step(record, other, others, [0, 1, 2]) == [3, 2, 1]


@pytest.mark.parametrize("number", [7, torch.full((1,), 7)])
def test_states_without_counts(record, number):
    """A file in which only the groups count: their number holds for the parameters that have a state."""
    params, opt = made()
    step(record, opt, params, [0, 1])
    saved = copy.deepcopy(opt.state_dict())
    for s in saved["state"].values():
        s.pop("step", None)
    saved["param_groups"][0]["step"] = number
    others, other = made()
    other.load_state_dict(saved)
    assert step(record, other, others, [0, 1, 2]) == [8, 8, 1]


def test_a_state_that_is_dropped_begins_again(record):
    params, opt = made()
    for _ in range(3):
        step(record, opt, params, [0, 1, 2])
    del opt.state[params[1]]
    assert step(record, opt, params, [0, 1, 2]) == [4, 1, 4]


def test_groups_that_change(record):
    """Parameters and groups that are added later begin with 1, and do not disturb the others."""
    params, opt = made(2)
    for _ in range(3):
        step(record, opt, params, [0, 1])
    more = [torch.nn.Parameter(torch.zeros(4)) for _ in range(2)]
    opt.add_param_group(dict(params=more[:1]))
    opt.param_groups[0]["params"].insert(0, more[1])
    assert step(record, opt, params + more, [0, 1, 2, 3]) == [4, 4, 1, 1]
    del opt.param_groups[0]["params"][1]
    params[0].grad = None
    assert step(record, opt, params[1:] + more, [0, 1, 2]) == [5, 2, 2]


def test_places_of_steps_refused_by_the_library():
    """Before any device call (the addresses are never read: sizes are 0 wherever a call is not refused)."""
    from allreduce_compatible_gradient_gb300 import _binding, _build
    _build.build_library()
    L = _binding.lib()
    P, N = ctypes.c_void_p * 2, ctypes.c_int64 * 2
    t, n, fake = P(None, None), N(0, 0), 1 << 20

    def step(at, counts=fake):
        return L.gq_adamw_step_places(2, t, 0, t, 0, t, t, None, n, 1, counts, 1e-3, 0.9, 0.999, 1e-8, 0.1, None, -1.0,
                                      0, 0, 0, None, at, None)
    assert step(None) == step(N(0, 0)) == step(N(5, (1 << 31) - 1)) == step(None, None) == 0
    for bad in (N(-1, 0), N(0, -1), N(0, 1 << 31), N((1 << 63) - 1, 0)):
        assert step(bad) == 1
    assert step(N(0, 0), None) == 1


def test_states_made_again(record):
    """make_states() for a dropped state, with gradients enabled: the others' counts stay."""
    params, opt = made()
    step(record, opt, params, [0, 1, 2])
    del opt.state[params[1]]
    opt.make_states()
    assert step(record, opt, params, [0, 1, 2]) == [2, 1, 2]
