"""AdamW as a torch optimizer over gq_adamw_step: one launch for all parameters, states in fp32 or in 8 bits.

8-bit states take 2.1 bytes a parameter instead of 8.  They, and bf16 parameters, are rounded at random
without bias by default (random=False: to nearest).  The words are those of (key, step, tensor, element) with a
key of the optimizer's own that no gradient and no MlpBlock8 draws from.  The step is the number of the tensor's
own steps; the tensor's number is given to it in its first one and kept with its state, whichever others have a
gradient later.  Words do not depend on the rank: data-parallel replicas that make the same steps stay equal bit
for bit.  `seed` (below 2^31) tells the optimizers of one program apart, where it has several.
"""
from __future__ import annotations

from array import array
from typing import NamedTuple

import torch

from . import _optimizer as ops


class _Counts(NamedTuple):
    """The numbers of steps that a group and, behind its own, each of its parameters have made: one tensor, on the
    device for captured steps, else over `host`'s memory, with its views, of which the states hold theirs; and the
    parameters' numbers."""

    counts: torch.Tensor
    host: array | None
    own: torch.Tensor
    steps: list
    places: list


class AdamW(torch.optim.Optimizer):
    """Decoupled weight decay (Loshchilov, Hutter, arXiv 1711.05101), as torch.optim.AdamW: a parameter's bias is
    corrected by the number of its own steps, those in which it had a gradient.

    states: "8bit" or "f32".  max_norm: gradients are clipped to this norm over all of them, and a step whose
    gradients hold a NaN, an infinity or a magnitude above 1.8e19 changes nothing (it still counts).
    capturable: the numbers of steps are kept on the device, so that step() can be captured into a graph and
    replayed (the states have to be there: make a step, or call make_states(), before); without it a capture is
    refused.  A captured step keeps the learning rate and the other settings of its capture, and works on the
    states that were there: capture again after changing a setting or load_state_dict().  Parameters are float32
    or bfloat16; those without a gradient are passed over.  A group's parameters lie on one GPU, with max_norm
    those of all groups."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, states="8bit",
                 max_norm=None, random=True, seed=0, capturable=False):
        if states not in ("8bit", "f32"):
            raise ValueError("states must be '8bit' or 'f32'")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError("betas must be at least 0 and below 1")
        if not eps >= 0.0 or (max_norm is not None and not max_norm >= 0.0):
            raise ValueError("eps and max_norm must not be negative")
        if not 0 <= seed < 1 << 31:
            raise ValueError("seed must be a number below 2^31")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, step=0,
                                      states=states))
        self.max_norm, self.random, self.seed, self.capturable = max_norm, random, seed, capturable
        self._forget()

    @property
    def key(self) -> int:
        """The key of the random words: between those of MlpBlock8's seeds and of its unnamed blocks."""
        return (1 << 64) - (1 << 33) + self.seed

    def __getstate__(self):
        own = ("max_norm", "random", "seed", "capturable")
        return {**super().__getstate__(), **{k: self.__dict__[k] for k in own}}

    def __setstate__(self, state):  # also of a load_state_dict()
        super().__setstate__(state)
        self._forget()

    def _forget(self):
        """What is kept beside the states is made anew from them."""
        self._kept, self._next = {}, None
        for index, group in enumerate(self.param_groups):
            states = [self.state[p] for p in group["params"] if self.state.get(p)]
            for s in states:  # of a file from before parameters counted
                s.setdefault("step", torch.tensor(int(group["step"]), device="cpu"))
            if states:
                self._counts(index, group)

    def make_states(self) -> None:
        """States of zeros for the parameters that have none, and with `capturable` the steps' numbers on the
        device."""
        for index, group in enumerate(self.param_groups):
            for p in group["params"]:
                self._state(p, group)
            if group["params"]:
                self._counts(index, group)

    def _counts(self, index, group):
        """A group's _Counts, as its states have them."""
        params, kept = group["params"], self._kept.get(index)
        device = params[0].device if self.capturable else torch.device("cpu")
        states = [self.state.get(p) for p in params]
        if (kept is None or kept.counts.device != device or len(kept.steps) != 1 + len(params)
                or self.capturable and group["step"] is not kept.own
                or any(s and s.get("step", v) is not v for s, v in zip(states, kept.steps[1:]))):
            self._not_captured()
            numbers = [int(group["step"]), *(int(s["step"]) if s and "step" in s else 0 for s in states)]
            host = None if self.capturable else array("q", numbers)
            counts = (torch.tensor(numbers, dtype=torch.int64, device=device) if host is None
                      else torch.frombuffer(host, dtype=torch.int64))
            kept = self._kept[index] = _Counts(counts, host, counts[:1], list(counts), [None] * len(numbers))
            if self.capturable:
                group["step"] = kept.own
            for s, v in zip(states, kept.steps[1:]):
                if s and "step" in s:
                    s["step"] = v
        for k, s in enumerate(states, 1):
            if s and "step" not in s:  # a new state, perhaps in the place of a dropped one
                kept.steps[k].zero_()
                kept.places[k] = None
                s["step"] = kept.steps[k]
        return kept

    def _place(self, s):
        """The number of the parameter of a state."""
        if "place" not in s:
            if self._next is None:
                self._next = 1 + max((int(v["place"]) for v in self.state.values() if "place" in v), default=-1)
            s["place"] = torch.tensor(self._next, device="cpu")
            self._next += 1
        return int(s["place"])

    @staticmethod
    def _add(kept, at, by):
        """counts[at] += by, on the device in as many launches as there are runs."""
        if kept.host is not None:
            for k in at:
                kept.host[k] += by
            return
        if len(at) == len(kept.steps):
            kept.counts.add_(by)
            return
        at = sorted(at)
        begin = 0
        for i in range(1, len(at) + 1):
            if i == len(at) or at[i] != at[i - 1] + 1:
                kept.counts[at[begin]:at[i - 1] + 1].add_(by)
                begin = i

    @staticmethod
    def _captured():
        return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()

    def _not_captured(self):
        # a graph would make them again, as zeros, at every replay
        if self._captured():
            raise RuntimeError("states are made before a step is captured: make a step, or call make_states()")

    def _state(self, p, group):
        s = self.state[p]
        if not s:
            self._not_captured()
            if group["states"] == "8bit":
                s.update(zip(("m", "v", "exps"), ops.gq_adamw_state(p.numel(), p.device)))
            else:
                s.update((k, torch.zeros(p.shape, dtype=torch.float32, device=p.device)) for k in ("m", "v"))
        return s

    def _norm(self, grads):
        """Over gradients of either type."""
        kinds = {}
        for g in grads:
            kinds.setdefault(g.dtype, []).append(g)
        first, *others = [ops.gq_tensors_norm(v) for v in kinds.values()]
        return torch.hypot(first, *others) if others else first

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if not self.capturable and self._captured():
            raise RuntimeError("a captured step would repeat its number at every replay: it needs capturable=True")
        calls, grads = [], []
        for index, group in enumerate(self.param_groups):
            some, lists, params, kept = [], {}, group["params"], self._kept.get(index)
            fits = kept is not None and len(kept.steps) == 1 + len(params)
            for k, p in enumerate(params, 1):
                g = p.grad
                if g is None:
                    continue
                if g.is_sparse:
                    raise RuntimeError("sparse gradients are not supported")
                g = g.contiguous()
                s = self._state(p, group)
                fits = fits and s.get("step") is kept.steps[k]
                grads.append(g)
                some.append((k, p, g, s))
            if not some:
                continue
            if not fits or self.capturable and (group["step"] is not kept.own or kept.own.device != grads[-1].device):
                kept = self._counts(index, group)
            steps = kept.host
            for entry in some:
                k, p, g, s = entry
                # a call's tensors are of one type, their states of one kind, and the host counts for all of them
                kind = p.dtype, g.dtype, "exps" in s, None if steps is None else steps[k] + 1
                lists.setdefault(kind, []).append(entry)
            # (parameters that are new get their numbers call by call, so that those of a call follow one another)
            for entries in lists.values():
                for k, _, _, s in entries:
                    if kept.places[k] is None:
                        kept.places[k] = self._place(s)
                places = [kept.places[entry[0]] for entry in entries]
                if places != sorted(places):
                    entries.sort(key=lambda entry: kept.places[entry[0]])
            calls.append((group, kept, lists))
        if not calls:
            return loss
        norm = None if self.max_norm is None else self._norm(grads)
        for group, kept, lists in calls:
            own = (0,)
            for (_, _, eight, step), entries in lists.items():
                at, params, gradients, states = zip(*entries)
                counted = own + at
                self._add(kept, counted, 1)
                try:
                    ops.gq_adamw_step_places(
                        params, gradients,
                        [(s["m"], s["v"], s["exps"]) if eight else (s["m"], s["v"]) for s in states],
                        step or kept.counts, [kept.places[k] for k in at], lr=group["lr"], betas=group["betas"],
                        eps=group["eps"], weight_decay=group["weight_decay"], norm=norm, max_norm=self.max_norm,
                        seed=self.key if self.random else None, step_places=None if step else at)
                except Exception:  # refused: these have made no step
                    self._add(kept, counted, -1)
                    raise
                own = ()
            if not self.capturable:
                group["step"] = int(group["step"]) + 1
        return loss

    def load_state_dict(self, state_dict) -> None:
        super().load_state_dict(state_dict)
        # torch gives floating-point parameters' states their type: bytes, and fp32 moments of bf16 parameters,
        # are taken as they are
        old = [i for group in state_dict["param_groups"] for i in group["params"]]
        new = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(old, new):
            if i in state_dict["state"]:
                self.state[p] = {k: v.detach().to("cpu" if k in ("place", "step") else p.device, copy=True)
                                 for k, v in state_dict["state"][i].items()}
        self._forget()
