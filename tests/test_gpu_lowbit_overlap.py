"""Tensors of a step that share memory: their updates would meet in it, and the result would be that of whichever
comes last."""
import pytest

from gpu_common import gq_module

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gq():
    return gq_module()


def pair(n):
    return torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")


def test_overlapping_parameters_and_states(gq):
    flat = torch.ones(1000, device="cuda")
    g = torch.ones(300, device="cuda")
    ours = [gq.gq_adamw_state(300) for _ in range(2)]
    step = gq.gq_adamw_step
    for a, b in ((0, 0), (0, 299), (299, 0), (100, 200), (700, 699)):
        with pytest.raises(ValueError, match="twice"):
            step([flat[a:a + 300], flat[b:b + 300]], [g, g], ours, 1)
    m = torch.zeros(1000, device="cuda")
    for a, b, c, d in ((0, 300, 299, 700), (0, 299, 600, 700), (0, 300, 600, 601)):
        with pytest.raises(ValueError, match="twice"):
            step([flat[:300], flat[300:600]], [g, g], [(m[a:a + 300], m[b:b + 300]), (m[c:c + 300], m[d:d + 300])], 1)
    with pytest.raises(ValueError, match="twice"):  # a state in a parameter's place
        step([flat[:300]], [g], [(flat[200:500], m[:300])], 1)
    one, other = ours
    for shared in (gq.Adam8(other.m, other.v, one.exps), gq.Adam8(other.m, one.v, other.exps),
                   gq.Adam8(one.m, other.v, other.exps), gq.Adam8(other.m, other.m, other.exps)):
        with pytest.raises(ValueError, match="twice"):
            step([flat[:300], flat[300:600]], [g, g], [one, shared], 1)
    assert (flat == 1).all() and not any(t.any() for s in ours for t in s)
    # side by side, without elements, gradients that are shared: as they are
    step([flat[:300], flat[300:600], flat[10:10]], [g, g, g[:0]],
         [(m[:300], m[300:600]), (m[600:900], torch.zeros(300, device="cuda")), pair(0)], 1)
    assert (flat[:600] != 1).all() and (flat[600:] == 1).all()


def test_overlapping_outputs(gq):
    states = [gq.gq_adamw_state(100) for _ in range(2)]
    flat = torch.ones(1000, device="cuda")
    at = lambda k: flat[k:k + 100]  # noqa: E731
    for x, r in (((0, 99), (200, 300)), ((0, 100), (199, 300)), ((0, 100), (200, 200)), ((0, 100), (100, 300))):
        with pytest.raises(ValueError, match="twice"):
            gq.gq_adamw_values(states, out=([at(k) for k in x], [at(k) for k in r]))
    assert (flat == 1).all()
    gq.gq_adamw_values(states, out=([at(0), at(100)], [at(200), at(300)]))
    assert not flat[:400].any() and (flat[400:] == 1).all()
