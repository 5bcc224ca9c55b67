"""Which random words the optimizer asks for, on a machine without a GPU: its calls are recorded in place of the
native entry point."""
import copy
import ctypes
import io

import pytest

torch = pytest.importorskip("torch")


class Recorder:
    """Stands for the native module: what each call gives to each parameter."""

    def __init__(self):
        self.calls = []

    def tensors_norm(self, tensors, ws):
        return torch.ones(1)

    def adamw_step(self, params, grads, states, step, *rest):
        first = rest[8]
        places = rest[9] if len(rest) > 9 and rest[9] is not None else range(len(params))
        for p, k in zip(params, places):
            self.calls.append((p, int(step), first + k))


@pytest.fixture
def record(monkeypatch):
    from allreduce_compatible_gradient_gb300 import _activations
    recorder = Recorder()
    monkeypatch.setattr(_activations, "_native", recorder)
    return recorder


def made(*groups, **kw):
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    params = [[torch.nn.Parameter(torch.zeros(4, dtype=t)) for t in types] for types in groups]
    return params, AdamW([dict(params=v) for v in params], **kw)


def step(opt, params, which):
    for p in params:
        p.grad = torch.ones_like(p) if any(p is q for q in which) else None
    opt.step()


def test_alternating_groups_share_no_words(record):
    """Two groups trained in turn, and then together: no two updates of different parameters have the same step and
    row of words."""
    (a, b), opt = made([torch.float32] * 2, [torch.float32] * 3)
    for which in (a, b, a + b, a[:1] + b[2:], b, a):
        step(opt, a + b, which)
    seen = {}
    for p, number, row in record.calls:
        assert seen.setdefault((number, row), p) is p
    assert len(record.calls) == 2 + 3 + 5 + 2 + 3 + 2


def test_rows_do_not_depend_on_the_gradients_there(record):
    """A parameter keeps its row, whichever others have a gradient; types are numbered one after the other as they
    appear in a group."""
    f, h = torch.float32, torch.bfloat16
    (a, b), opt = made([f, h, f, h], [h, f])
    every = a + b
    step(opt, every, every)
    rows = {id(p): row for p, _, row in record.calls}
    assert [rows[id(p)] for p in every] == [0, 2, 1, 3, 4, 5]
    for which in (every[1:], every[::2], every[3:4]):
        del record.calls[:]
        step(opt, every, which)
        assert len(record.calls) == len(which)
        assert all(rows[id(p)] == row for p, _, row in record.calls)


@pytest.mark.parametrize("how", ["file", "deep copy", "state of its own", "group added"])
def test_rows_are_kept(record, how):
    """Numbers given in the order of the first gradients go with the states."""
    (a,), opt = made([torch.float32] * 4)
    for which in (a[2:3], a[:1] + a[3:]):
        step(opt, a, which)
    late = torch.nn.Parameter(torch.zeros(3))
    if how == "deep copy":
        opt = copy.deepcopy(opt)
        a = opt.param_groups[0]["params"]
    elif how == "group added":
        opt.add_param_group(dict(params=[late]))
    else:
        saved = opt.state_dict()
        if how == "file":
            f = io.BytesIO()
            torch.save(saved, f)
            f.seek(0)
            saved = torch.load(f)
        (a,), opt = made([torch.float32] * 4)
        step(opt, a, a)  # its own numbers give way
        opt.load_state_dict(saved)
    if how != "group added":
        opt.add_param_group(dict(params=[late]))
    del record.calls[:]
    step(opt, [*a, late], [*a, late])
    rows = {id(p): row for p, _, row in record.calls}
    assert [rows[id(p)] for p in (*a, late)] == [1, 3, 0, 2, 4]


def test_states_without_numbers(record):
    """A file from before the numbers: its parameters get some in the order of the calls."""
    (a,), opt = made([torch.float32] * 3)
    step(opt, a, a)
    saved = copy.deepcopy(opt.state_dict())
    for s in saved["state"].values():
        s.pop("place", None)
    (b,), other = made([torch.float32] * 3)
    other.load_state_dict(saved)
    del record.calls[:]
    step(other, b, b[1:])
    step(other, b, b)
    rows = {}
    for p, _, row in record.calls:
        assert rows.setdefault(id(p), row) == row
    assert [rows[id(p)] for p in b] == [2, 0, 1]


def test_a_state_that_is_dropped(record):
    (a,), opt = made([torch.float32] * 3)
    step(opt, a, a)
    del opt.state[a[1]]
    step(opt, a, a)
    last = [row for p, _, row in record.calls[3:]]
    assert sorted(last) == [0, 2, 3] and record.calls[5][0] is a[1]


def test_places_refused_by_the_library():
    """Before any device call (the addresses are never read: sizes are 0 wherever a call is not refused)."""
    from allreduce_compatible_gradient_gb300 import _binding, _build
    _build.build_library()
    L = _binding.lib()
    P, N = ctypes.c_void_p * 2, ctypes.c_int64 * 2
    t, n = P(None, None), N(0, 0)

    def step(places, first=0):
        return L.gq_adamw_step_places(2, t, 0, t, 0, t, t, None, n, 1, None, 1e-3, 0.9, 0.999, 1e-8, 0.1, None, -1.0, 0,
                                      0, first, places, None, None)
    top = (1 << 30) - 1
    for good, first in ((None, 0), (N(0, 1), 0), (N(5, top), 0), (N(0, top - 7), 7), (None, top - 1)):
        assert step(good, first) == 0
    for bad, first in ((N(0, 0), 0), (N(1, 0), 0), (N(-1, 0), 0), (N(0, top + 1), 0), (N(0, top - 6), 7),
                       (N(0, (1 << 63) - 1), 0), (None, top), (None, (1 << 63) - 1), (N(0, 1), (1 << 63) - 1)):
        assert step(bad, first) == 1
