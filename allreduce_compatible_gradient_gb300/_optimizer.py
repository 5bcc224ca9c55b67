"""The AdamW step over many tensors at once and the norm of all gradients (include/gq.h, the section on the
optimizer's step): argument checks and marshalling over libgq.so.  `adamw.AdamW` is a torch optimizer over
them.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _activations as _acts
from ._activations import _on
from ._binding import lib


class Adam8(NamedTuple):
    """The two moments of a tensor of n elements in 8 bits, with N = round_up(n, 32): e4m3 codes of the first
    (N bytes), codes of the second's root (N bytes), and the exponent bytes of every 32 elements (N / 32 pairs).
    All zeros is a state of zeros."""

    m: torch.Tensor
    v: torch.Tensor
    exps: torch.Tensor


def gq_adamw_state(numel: int, device="cuda") -> Adam8:
    """An 8-bit state of zeros for a tensor of numel elements."""
    if numel < 0:
        raise ValueError("numel must not be negative")
    n = (numel + 31) // 32 * 32
    m, v = (torch.zeros(n, dtype=torch.uint8, device=device) for _ in range(2))
    return Adam8(m, v, torch.zeros((n // 32, 2), dtype=torch.uint8, device=device))


def gq_tensors_norm_workspace_bytes(count: int) -> int:
    return lib().gq_tensors_norm_workspace_bytes(count)


def gq_tensors_norm(tensors, ws=None, stream=None) -> torch.Tensor:
    """The square root of the sum of the squares of all elements of all tensors (a list of contiguous float32
    or bfloat16 tensors, of one type): one float32 number on the device, infinite or a NaN where a magnitude is above
    1.8e19 (whose square is no fp32 number) or not finite.  Magnitudes below 1.1e-19 lose digits, those below 2.6e-23
    count as 0."""
    if stream is not None:
        return _on(stream, gq_tensors_norm, tensors, ws)
    return _acts._native.tensors_norm(tensors, ws)


def gq_adamw_step(params, grads, states, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                  norm=None, max_norm=None, seed=None, first=0, stream=None) -> None:
    """One AdamW step, in place, on lists of contiguous tensors, of which parameters and states share no memory.

    params and grads: float32 or bfloat16 (all of a list of one type); states: an Adam8 or a pair of float32
    tensors (first and second moment) for each, all of one kind.  step: the step's number from 1 on, or an
    int64 tensor on the device that holds it (captured graphs).  norm: gq_tensors_norm's result; a step whose
    norm is not finite changes nothing, and with max_norm the gradients are scaled by
    min(1, max_norm / (norm + 1e-6)).  seed: 8-bit states and bfloat16 parameters are rounded at random without
    bias, else to nearest; `first` is the number of the first tensor where a program makes several calls per
    step, so that no two tensors share random words."""
    if stream is not None:
        return _on(stream, gq_adamw_step, params, grads, states, step, lr, betas, eps, weight_decay, norm,
                   max_norm, seed, first)
    beta1, beta2 = betas
    return _acts._native.adamw_step(params, grads, states, step, lr, beta1, beta2, eps, weight_decay, norm,
                                    max_norm, seed, first, None, None)


def gq_adamw_step_places(params, grads, states, step, places, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                         weight_decay=1e-2, norm=None, max_norm=None, seed=None, first=0, step_places=None,
                         stream=None) -> None:
    """gq_adamw_step for lists that leave out some of a program's tensors.  places: a number for each tensor, in
    ascending order, counted from `first`: its random words are those of its number, whichever others are there.
    step_places: for a `step` on the device that holds several numbers, the place of each tensor's."""
    if stream is not None:
        return _on(stream, gq_adamw_step_places, params, grads, states, step, places, lr, betas, eps,
                   weight_decay, norm, max_norm, seed, first, step_places)
    if places is None:
        raise TypeError("places must be a list or a tuple")
    beta1, beta2 = betas
    return _acts._native.adamw_step(params, grads, states, step, lr, beta1, beta2, eps, weight_decay, norm,
                                    max_norm, seed, first, places, step_places)


def gq_adamw_values(states, out=None, out_dtype=torch.bfloat16, stream=None):
    """(first moments, roots of the second moments): the values of 8-bit states, two lists of tensors of
    out_dtype (float32 or bfloat16) with the states' padding, or the two lists `out`, each tensor with its
    parameter's elements."""
    if stream is not None:
        return _on(stream, gq_adamw_values, states, out, out_dtype)
    if out is None:
        out = tuple([torch.empty(s.m.shape, dtype=out_dtype, device=s.m.device) for s in states]
                    for _ in range(2))
    _acts._native.adamw_values(states, *out)
    return out
