"""The random words of the optimizer's parameters: none share any, whichever have a gradient."""
import pytest

import lowbit_ref as ref
from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gq():
    return gq_module()


def test_alternating_groups_round_apart(gq):
    """Two groups of equal values and gradients, updated in turn: rounding tells them apart."""
    from allreduce_compatible_gradient_gb300.adamw import AdamW
    g = torch.Generator(device="cuda").manual_seed(1)
    x, d = (torch.randn(4096, generator=g, device="cuda") for _ in range(2))
    a, b = (torch.nn.Parameter(x.clone()) for _ in range(2))
    opt = AdamW([dict(params=[a]), dict(params=[b])])
    for p, q in ((a, b), (b, a)):
        p.grad, q.grad = d, None
        opt.step()
    # of 4,096 codes, each at one of 2^16 places between two: some differ
    assert not torch.equal(opt.state[a]["m"], opt.state[b]["m"])
    assert not torch.equal(opt.state[a]["v"], opt.state[b]["v"])


@pytest.mark.parametrize("seed", [0, 2 ** 63 + 11])
def test_words_of_places(gq, seed):
    """Codes bit for bit from the words of their places.  The first step from zeros with beta1 = 1/2, beta2 = 3/4:
    m = g / 2, root |g| / 2, exact in fp32 for small integers times powers of two."""
    sizes, places, step = [40, 1000, 0, 33], [0, 5, 6, (1 << 29) - 8], 2 ** 40 + 3
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.randint(-2047, 2048, (n,), generator=g, device="cuda").float() for n in sizes]
    params = [torch.zeros(n, device="cuda") for n in sizes]
    states = [gq.gq_adamw_state(n) for n in sizes]
    gq.gq_adamw_step_places(params, grads, states, step, places, betas=(0.5, 0.75), seed=seed, first=7)
    for d, s, k in zip(grads, states, places):
        n = d.numel()
        if n == 0:
            continue
        h = [ref.words(n, 3 * (7 + k) + j, seed, step, "cuda") for j in range(2)]
        qm, _, _ = ref.on_grid(d.double().abs() / 2, ref.E4M3_MOST, 3, -9, h[0], False)
        qr, _, _ = ref.on_grid(d.double().abs() / 2, ref.ROOT_MOST, 4, 0, h[1], True)
        out = tuple([torch.empty(n, device="cuda")] for _ in range(2))
        gq.gq_adamw_values([s], out=out)
        assert torch.equal(out[0][0].double(), torch.sign(d.double()) * qm) and torch.equal(out[1][0].double(), qr)


def test_places_refused(gq):
    p, d = ([torch.zeros(64, device="cuda") for _ in range(2)] for _ in range(2))
    s = [gq.gq_adamw_state(64) for _ in range(2)]
    for bad in ([0], [0, 0], [1, 0], [-1, 0], [0, 1 << 30], [0, 1 << 62], [0, 1, 2]):
        with pytest.raises(ValueError):
            gq.gq_adamw_step_places(p, d, s, 1, bad, seed=1)
    with pytest.raises(TypeError):
        gq.gq_adamw_step_places(p, d, s, 1, 5, seed=1)
    with pytest.raises(ValueError):
        gq.gq_adamw_step_places(p, d, s, 1, [0, 8], seed=1, first=(1 << 30) - 8)
    assert not any(t.any() for t in p)
