"""Which random words the layers over 8-bit checkpoints round with: no two roundings share any."""
import copy
import io
import os
import pickle
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    from allreduce_compatible_gradient_gb300.act8_layers import MlpBlock8
    return lambda **kw: MlpBlock8(8, 16, **kw)


def words(*blocks):
    return [b.words(layer) for b in blocks for layer in (0, 1)]


def test_every_layer_has_words_of_its_own(block):
    blocks = [block() for _ in range(5)]
    blocks += [copy.deepcopy(blocks[0]), copy.copy(blocks[0]), pickle.loads(pickle.dumps(blocks[0]))]
    f = io.BytesIO()
    torch.save(blocks[0], f)
    f.seek(0)
    blocks.append(torch.load(f, weights_only=False))
    blocks += [block(seed=s) for s in (0, 1, 2, 1 << 31, (1 << 62) - (1 << 32) - 1)]
    seeds = [seed for seed, _ in words(*blocks)]
    assert len(set(seeds)) == len(seeds)


def test_a_seed_names_the_words(block):
    assert words(block(seed=7)) == words(block(seed=7))


def test_words_are_not_those_of_gradients(block):
    """Whose seeds lie below 2^63."""
    assert all(1 << 63 <= seed < 1 << 64 for seed, _ in words(block(), block(seed=0), block(seed=3)))


def test_ranks_and_steps_have_words_of_their_own(block):
    b, seen = block(), set()
    for b.rank in (0, 1, 2, (1 << 16) - 1):
        for b.step in (0, 1, 2, 1000, (1 << 48) - 1):
            seen |= set(words(b))
    assert len(seen) == 2 * 4 * 5 and all(0 <= step < 1 << 64 for _, step in seen)


def test_the_rank_is_the_process_groups(block, monkeypatch):
    b = block()
    alone = words(b)
    monkeypatch.setattr(torch.distributed, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.distributed, "get_rank", lambda: 3)
    assert [step for _, step in words(b)] == [3 << 48] * 2
    b.rank = 0
    assert words(b) == alone


@pytest.mark.parametrize("kw,step", [(dict(seed=-1), 0), (dict(seed=1 << 62), 0), (dict(rank=-1), 0),
                                     (dict(rank=1 << 16), 0), (dict(), -1), (dict(), 1 << 48)])
def test_numbers_that_do_not_fit_are_refused(block, kw, step):
    b = block(**kw)
    b.step = step
    with pytest.raises(ValueError):
        b.words(0)


def test_the_examples_workers_have_words_of_their_own(monkeypatch):
    """Every forward pass of a training step with gradients, and the gradients' own rounding."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_mlp8 as example
    finally:
        sys.path.pop(0)
    seen, mean_seeds = [], []

    def forward(self, x):
        if torch.is_grad_enabled():
            seen.extend(self.words(layer) for layer in (0, 1))
        return x + torch.nn.functional.linear(torch.nn.functional.linear(x.float(), self.w1), self.w2)

    def mean(grads, q, p, scheme, s, seed, step, ws):
        mean_seeds.append(seed)
        return grads.mean(0)
    on_cpu = lambda make: lambda *a, device=None, **kw: make(*a, **kw)  # noqa: E731
    monkeypatch.setattr(example.MlpBlock8, "__init__", on_cpu(example.MlpBlock8.__init__))
    monkeypatch.setattr(example.MlpBlock8, "forward", forward)
    monkeypatch.setattr(example.gq, "gq_allreduce_mean", mean)
    monkeypatch.setattr(example.gq, "gq_workspace", lambda device: None)
    real = {name: getattr(torch, name) for name in ("empty", "randn")}
    for name, make in real.items():
        monkeypatch.setattr(torch, name, on_cpu(make))
    monkeypatch.setattr(torch.autograd, "grad",
                        lambda loss, params: [torch.zeros_like(p) for p in params])
    example.train(workers=3, steps=4, width=8, hidden=16, tokens=5)
    assert len(seen) == 3 * 4 * 2 * 2 and len(set(seen)) == len(seen)
    assert all(seed < 1 << 63 for seed in mean_seeds) and not {seed for seed, _ in seen} & set(mean_seeds)
