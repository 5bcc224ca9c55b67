"""gq_linear_wgrad_plan on a machine without a GPU: every step of every tile in one share."""
import ctypes
import random

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def plan():
    from allreduce_compatible_gradient_gb300 import _binding, _build
    _build.build_library()

    def call(rows, outs, cols, dtype=1, ld=None):
        p = (ctypes.c_int64 * 8)()
        r = _binding.lib().gq_linear_wgrad_plan(1 << 20, dtype, rows, outs, outs if ld is None else ld, cols, p)
        return r, list(p)
    return call


def test_random_sizes(plan):
    rng = random.Random(5)
    for _ in range(2000):
        rows, outs, cols = (int(2 ** rng.uniform(0, top)) for top in (16, 13, 13))
        dtype = rng.choice([0, 1])
        r, (th, tw, steps, shares, own, left, longest, chain) = plan(rows, outs, cols, dtype)
        assert r == 0 and (th, tw) in ((512, 256), (128, 128)) and chain == 96
        assert steps == (3 if dtype == 0 else 1) * -(-rows // 64)
        assert own * shares + left == -(-outs // th) * -(-cols // tw) and 0 <= left < shares
        most = steps if own else 0
        if left:
            most = max(most, min(steps, -(-left * steps // shares)))
        assert most / 2 <= longest <= max(most, 1)  # a share's piece may lie across two tiles


def test_refusals_and_no_rows(plan):
    assert plan(0, 64, 64) == (0, [0] * 8)
    for bad in (dict(rows=-1), dict(outs=0), dict(cols=0), dict(dtype=2), dict(rows=1 << 29)):
        assert plan(**{**dict(rows=64, outs=64, cols=64), **bad})[0] == 1, bad
    from allreduce_compatible_gradient_gb300 import _binding
    assert _binding.lib().gq_linear_wgrad_plan(1 << 20, 1, 64, 64, 64, 64, None) == 1
