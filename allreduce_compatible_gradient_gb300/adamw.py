"""AdamW as a torch optimizer over gq_adamw_step: one launch for all parameters, states in fp32 or in 8 bits.

8-bit states take 2.1 bytes a parameter instead of 8.  They, and bf16 parameters, are rounded at random
without bias by default (random=False: to nearest).  The words are those of (key, step, tensor, element) with a
key of the optimizer's own that no gradient and no MlpBlock8 draws from.  A tensor's number is given to it in its
first step and kept with its state, whichever others have a gradient later.  Words do not depend on the rank:
data-parallel replicas that make the same steps stay equal bit for bit.  `seed` (below 2^31) tells the
optimizers of one program apart, where it has several.
"""
from __future__ import annotations

import torch

from . import _optimizer as ops


class AdamW(torch.optim.Optimizer):
    """Decoupled weight decay (Loshchilov, Hutter, arXiv 1711.05101), as torch.optim.AdamW.

    states: "8bit" or "f32".  max_norm: gradients are clipped to this norm over all of them, and a step whose
    gradients hold a NaN or an infinity changes nothing (it still counts).  capturable: the number of the step
    is kept on the device, so that step() can be captured into a graph and replayed (the states have to be
    there: make a step, or call make_states(), before).  A captured step keeps the learning rate and the other
    settings of its capture, and works on the states that were there: capture again after changing a setting or
    load_state_dict().  Parameters are float32 or bfloat16; those without a
    gradient are passed over."""

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
        """Of the states, what is read from them once."""
        self._places, self._next = {}, None

    def _place(self, p):
        """The parameter's number."""
        place = self._places.get(p)
        if place is None:
            s = self.state[p]
            if "place" not in s:
                if self._next is None:
                    self._next = 1 + max((int(v["place"]) for v in self.state.values() if "place" in v), default=-1)
                s["place"] = torch.tensor(self._next, device="cpu")
                self._next += 1
            place = self._places[p] = int(s["place"])
        return place

    def make_states(self) -> None:
        """States of zeros for the parameters that have none, and with `capturable` the steps' numbers on the
        device."""
        for group in self.param_groups:
            for p in group["params"]:
                self._state(p, group)
            if self.capturable and group["params"]:
                self._number(group, group["params"][0].device)

    def _number(self, group, device):
        """The group's count of steps as a tensor on the device."""
        if not torch.is_tensor(group["step"]) or group["step"].device != device:
            self._not_captured()
            group["step"] = torch.full((1,), int(group["step"]), dtype=torch.int64, device=device)
        return group["step"]

    @staticmethod
    def _not_captured():
        # a graph would make them again, as zeros, at every replay
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("states are made before a step is captured: make a step, or call make_states()")

    def _state(self, p, group):
        s = self.state[p]
        if not s:
            self._not_captured()
            self._places.pop(p, None)
            if group["states"] == "8bit":
                s.update(zip(("m", "v", "exps"), ops.gq_adamw_state(p.numel(), p.device)))
            else:
                s.update((k, torch.zeros(p.shape, dtype=torch.float32, device=p.device)) for k in ("m", "v"))
        return ops.Adam8(s["m"], s["v"], s["exps"]) if "exps" in s else (s["m"], s["v"])

    def _norm(self, grads):
        """Over gradients of either type."""
        norms = [ops.gq_tensors_norm(v) for v in ([g for g in grads if g.dtype == t]
                                                  for t in (torch.float32, torch.bfloat16)) if v]
        return norms[0] if len(norms) == 1 else torch.stack(norms).norm(dim=0)

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        calls, grads = [], []
        for group in self.param_groups:
            lists = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                if p.grad.is_sparse:
                    raise RuntimeError("sparse gradients are not supported")
                g = p.grad.contiguous()
                grads.append(g)
                state = self._state(p, group)
                # a call's tensors are of one type, and their states of one kind
                lists.setdefault((p.dtype, g.dtype, len(state)), []).append((p, g, state))
            # (parameters that are new get their numbers call by call, so that those of a call follow one another)
            lists = [sorted(((self._place(p), p, g, s) for p, g, s in entries), key=lambda entry: entry[0])
                     for entries in lists.values()]
            if lists:
                calls.append((group, lists))
        if not calls:
            return loss
        norm = None if self.max_norm is None else self._norm(grads)
        for group, lists in calls:
            if self.capturable:
                self._number(group, grads[0].device).add_(1)
            else:
                group["step"] = int(group["step"]) + 1
            for entries in lists:
                places, params, gradients, states = map(list, zip(*entries))
                ops.gq_adamw_step_places(params, gradients, states, group["step"], places, lr=group["lr"],
                                         betas=group["betas"], eps=group["eps"],
                                         weight_decay=group["weight_decay"], norm=norm, max_norm=self.max_norm,
                                         seed=self.key if self.random else None)
        return loss

    def load_state_dict(self, state_dict) -> None:
        super().load_state_dict(state_dict)
        # torch gives floating-point parameters' states their type: bytes, and fp32 moments of bf16 parameters,
        # are taken as they are
        old = [i for group in state_dict["param_groups"] for i in group["params"]]
        new = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(old, new):
            if i in state_dict["state"]:
                self.state[p] = {k: v.detach().to("cpu" if k == "place" else p.device, copy=True)
                                 for k, v in state_dict["state"][i].items()}
        self._forget()
