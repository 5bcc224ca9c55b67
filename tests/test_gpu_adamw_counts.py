"""Parameters whose gradients come late, or not in every step: their bias is corrected by the number of their own
updates, as in torch's AdamW."""
import copy

import pytest

import lowbit_ref as ref
from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SHAPES = ((64, 33), (33,), (5,), (5000,))
# parameters with a gradient in step k: one from the tenth on, one in every other step
WHICH = [[i for i in range(4) if (i != 1 or k >= 9) and (i != 2 or k % 2 == 0)] for k in range(20)]


@pytest.fixture(scope="module")
def gq():
    return gq_module()


def parameters():
    g = torch.Generator(device="cuda").manual_seed(1)
    return [torch.nn.Parameter(torch.randn(s, generator=g, device="cuda")) for s in SHAPES]


def with_gradients(params, seed, which):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i, p in enumerate(params):
        d = torch.randn(p.shape, generator=g, device="cuda") * 0.1
        p.grad = d if i in which else None


def near(ours, theirs, steps=20):
    """As beside torch's AdamW in fp64 with gradients in every step: a step's rounding is within 3 units of fp32 of
    the parameter and 32 of lr (bias corrections in fp32, where the device counts, within 2^-20 of lr)."""
    for p, q in zip(ours, theirs):
        off = (p.double() - q.double()).abs()
        assert (off <= steps * (3 * 2.0 ** -24 * q.double().abs() + 1e-2 * 2.0 ** -19)).all(), off.max()


@pytest.mark.parametrize("capturable", [False, True])
def test_late_parameters_follow_torch(gq, capturable):
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    ours = parameters()
    theirs = [torch.nn.Parameter(p.detach().double()) for p in ours]
    a = AdamW(ours, lr=1e-2, weight_decay=0.1, states="f32", capturable=capturable)
    b = torch.optim.AdamW(theirs, lr=1e-2, weight_decay=0.1)
    for k, which in enumerate(WHICH):
        with_gradients(ours, k, which)
        for p, q in zip(ours, theirs):
            q.grad = None if p.grad is None else p.grad.double()
        a.step()
        b.step()
    near(ours, theirs)
    assert [int(a.state[p]["step"]) for p in ours] == [int(b.state[q]["step"]) for q in theirs]


def test_first_update_is_lr(gq):
    """Betas as they are by default, 1,000 steps without it: the late parameter's first update is lr along the
    gradient's sign."""
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    p, q = (torch.nn.Parameter(torch.zeros(64, device="cuda")) for _ in range(2))
    opt = AdamW([p, q], lr=1e-3, weight_decay=0.0)
    p.grad = torch.ones(64, device="cuda")
    for _ in range(1000):
        opt.step()
    q.grad = torch.full((64,), -0.5, device="cuda")
    opt.step()
    assert ((q - 1e-3).abs() <= 1e-8).all()


def test_captured_steps_with_others_between(gq):
    """A captured step of some parameters, and eager ones of others between its replays: each counts its own, bit
    for bit as without a graph."""
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    ours, theirs = parameters(), parameters()
    a, b = (AdamW(p, lr=1e-2, max_norm=0.5, capturable=True) for p in (ours, theirs))
    a.make_states()
    b.make_states()
    with_gradients(ours, 1, [0, 2])
    held = [p.grad for p in ours]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for k in range(6):
        graph.replay()
        with_gradients(theirs, 1, [0, 2])
        b.step()
        for params, opt in ((ours, a), (theirs, b)):
            with_gradients(params, 10 + k, [1, 2] if k % 2 else [1, 3])
            opt.step()
        assert all(torch.equal(p, q) for p, q in zip(ours, theirs))
    del held
    assert [int(a.state[p]["step"]) for p in ours] == [int(b.state[q]["step"]) for q in theirs] == [6, 6, 9, 3]


def test_captured_after_loading_and_copying(gq):
    """Counts that come from a file or a copy are there when the next step is a captured one."""
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    ours = parameters()
    a = AdamW(ours, capturable=True)
    with_gradients(ours, 1, range(4))
    a.step()
    a.step()
    theirs = parameters()
    b = AdamW(theirs, capturable=True)
    b.load_state_dict(a.state_dict())
    c = copy.deepcopy(a)
    twins = c.param_groups[0]["params"]
    with torch.no_grad():
        for p, q in zip(ours, theirs):
            q.copy_(p)
    for params, opt in ((theirs, b), (twins, c)):
        with_gradients(params, 1, range(4))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step()
        graph.replay()
        graph.replay()
    a.step()
    a.step()
    for params in (theirs, twins):
        assert all(torch.equal(p, q) for p, q in zip(ours, params))


@pytest.mark.parametrize("eight", [False, True])
def test_places_of_steps(gq, eight):
    """A step whose tensors count by themselves on the device, against calls of one tensor each."""
    sizes, places, at = [500, 33, 0, 4097], [1, 2, 4, 6], [6, 1, 2, 1]
    counts = torch.tensor([9, 1, 50, 9, 9, 9, 1000], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    params = [torch.randn(n, generator=g, device="cuda") for n in sizes]
    grads = [torch.randn(n, generator=g, device="cuda") for n in sizes]

    def states():
        return [gq.gq_adamw_state(n) if eight else tuple(torch.zeros(n, device="cuda") for _ in range(2))
                for n in sizes]

    ours, theirs, one, other = [p.clone() for p in params], [p.clone() for p in params], states(), states()
    gq.gq_adamw_step_places(ours, grads, one, counts, places, seed=3, first=2, step_places=at)
    for p, d, s, k, i in zip(theirs, grads, other, places, at):
        gq.gq_adamw_step([p], [d], [s], counts[i:i + 1], seed=3, first=2 + k)
    for p, q, s, t in zip(ours, theirs, one, other):
        assert torch.equal(p, q) and all(torch.equal(x, y) for x, y in zip(s, t))

    def refused(step, at):
        with pytest.raises(ValueError):
            gq.gq_adamw_step_places(ours, grads, one, step, places, step_places=at)

    for bad in (counts[:6], counts[:0], counts.int(), counts.cpu(), torch.stack([counts, counts], 1)[:, 0], 5):
        refused(bad, at)
    for bad in ([6, 1, 2], [6, 1, 2, 7], [6, 1, 2, -1], None):
        refused(counts, bad)
    with pytest.raises(ValueError):
        gq.gq_adamw_step(ours, grads, one, counts)


def test_first_steps_of_late_parameters_by_hand(gq):
    """The definition, with one number a tensor: a tensor's t is its own."""
    g = torch.Generator(device="cuda").manual_seed(6)
    old = [torch.randn(300, generator=g, device="cuda") for _ in range(2)]
    grads = [torch.randn(300, generator=g, device="cuda") for _ in range(2)]
    params = [p.clone() for p in old]
    states = [tuple(torch.zeros(300, device="cuda") for _ in range(2)) for _ in range(2)]
    gq.gq_adamw_step_places(params, grads, states, torch.tensor([1, 0, 1000], device="cuda"), [0, 1], lr=0.01,
                            step_places=[0, 2])
    for p, q, d, t in zip(params, old, grads, (1, 1000)):
        want, _, _ = ref.adamw(q, d, torch.zeros_like(q), torch.zeros_like(q), t, 0.01, (0.9, 0.999), 1e-8, 0.01)
        # the update is at most 3.2 lr here; expm1 of a rounded exponent leaves 1e-6 of it, fp32 the rest
        assert ((p.double() - want).abs() <= 4e-2 * (1e-6 + 40 * 2.0 ** -24) + 3 * 2.0 ** -24 * want.abs()).all()
