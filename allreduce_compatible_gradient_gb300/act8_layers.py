"""Transformer layers that keep their activations in 8 bits (torch modules over the activation
operators): layer norm + linear, GELU + linear, and the pre-norm MLP block made of the two.

Parameters are fp32 (or bf16, as their gradients then are); activations and their gradients are bf16 (or
fp32).  The forward pass keeps one 8-bit checkpoint per normalised input and one per GELU input, and
nothing else of their size: the checkpoint of the normalised rows serves both the layer norm's backward
pass and the weight gradient of the linear layer behind it, and GELU's backward pass rebuilds the second
linear layer's input.  They are saved tensors like any others: the backward pass frees them, and
saved-tensor hooks see them.  Where no backward pass will read one (under no_grad, or with nothing before
it that requires a gradient) it is not made.

Checkpoints are rounded at random without bias, with random words of (key, step, row, column) as
gq_quantize draws them for gradients.  An estimate made of several roundings is unbiased only where their
words are independent, so no two share any: every layer of every block has a key of its own, bit 63 of
which is set (gradients keep theirs clear by seeds below 2^63), and the rank of a data-parallel job is part
of the step.

With products="e4m3" the linear layers' products run in 8-bit floating point: inputs and gradients with an
exponent per 128 columns of a row, weights with one per 128 x 128 elements, put into it in every forward pass
and kept (1 byte an element) for the input's gradient.  Weight gradients stay bf16 products on the checkpoints.
Gradients are those of the products as if nothing were rounded (straight through).

Gradients are of the first order only: a second derivative (create_graph=True, then a backward pass
through the result) raises a RuntimeError.
"""
from __future__ import annotations

import itertools

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import _activations as ops
from . import _fp8 as fp8


def _rows(x):
    """x as a matrix that the operators take: a copy where its elements do not lie side by side, or where
    rows share their memory."""
    m = x.reshape(-1, x.shape[-1])
    return m if m.stride(1) == 1 and (m.shape[0] < 2 or m.stride(0) >= m.shape[1]) else m.contiguous()


def _product(y, weight, bias, e4m3):
    """y weight^T + bias, and what its backward pass reads of the weight in 8 bits."""
    if not e4m3:
        return torch.nn.functional.linear(y, weight.to(y.dtype), bias.to(y.dtype)), None
    w8 = fp8.gq_fp8_quantize(_rows(weight), tiles=True)
    return fp8.gq_fp8_linear(y, w8, bias=bias.float()), w8.data


def _input_gradient(d, weight, data):
    if data is None:
        return d @ weight.to(d.dtype)
    return fp8.gq_fp8_linear_dgrad(d, fp8.Fp8.of_data(data, *weight.shape, tiles=True))


class _NormLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, norm_weight, norm_bias, weight, bias, eps, seed, step, record=True, e4m3=False):
        y, _, rstd, act = ops.gq_layernorm_forward(_rows(x), norm_weight, norm_bias, eps, seed=seed, step=step,
                                                   checkpoint=record and any(ctx.needs_input_grad[:4]))
        out, w8 = _product(y, weight, bias, e4m3)
        ctx.save_for_backward(norm_weight, norm_bias, weight, rstd, act and act.data,
                              w8 if any(ctx.needs_input_grad[:3]) else None)
        ctx.shape = x.shape
        return out.view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        norm_weight, norm_bias, weight, rstd, data, w8 = ctx.saved_tensors
        d = _rows(dout)
        need = ctx.needs_input_grad
        dx = dnw = dnb = dweight = dbias = None
        act = None if data is None else ops.Act8.of_data(data, weight.shape[1])
        if need[3]:
            dweight, dbias = ops.gq_linear_wgrad(d, act, scale=norm_weight.float(), shift=norm_bias.float(),
                                                 need_bias=need[4])
        elif need[4]:
            dbias = d.sum(0, dtype=torch.float32)
        if any(need[:3]):
            dx, dnw, dnb = ops.gq_layernorm_backward(_input_gradient(d, weight, w8), norm_weight, rstd, act=act)
            dx = dx.view(ctx.shape)
        return dx, dnw, dnb, dweight, dbias, None, None, None, None, None


class _GeluLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, weight, bias, approximate, seed, step, record=True, e4m3=False):
        h, act = ops.gq_gelu_forward(_rows(u), approximate=approximate, seed=seed, step=step,
                                     checkpoint=record and any(ctx.needs_input_grad[:2]))
        out, w8 = _product(h, weight, bias, e4m3)
        ctx.save_for_backward(weight, act and act.data, w8 if any(ctx.needs_input_grad[:2]) else None)
        ctx.approximate, ctx.shape = approximate, u.shape
        return out.view(*u.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        weight, data, w8 = ctx.saved_tensors
        d = _rows(dout)
        need = ctx.needs_input_grad
        du = dweight = None
        if need[0] or need[1]:
            got = ops.gq_gelu_backward(_input_gradient(d, weight, w8), ops.Act8.of_data(data, weight.shape[1]),
                                       approximate=ctx.approximate, need_output=need[1])
            du, h = got if need[1] else (got, None)
            du = du.view(ctx.shape)
            if need[1]:
                # bf16 operands, fp32 sums: the gradient of an fp32 parameter is not rounded to bf16
                dweight = d.t() @ h if d.dtype == torch.float32 else torch.mm(d.t(), h, out_dtype=torch.float32)
        dbias = d.sum(0, dtype=torch.float32) if need[2] else None
        return du, dweight, dbias, None, None, None, None, None


_numbers = itertools.count()  # of the blocks of this process


class MlpBlock8(nn.Module):
    """x + W2 gelu(W1 norm(x) + b1) + b2 with 8-bit checkpoints.

    `step` numbers the training steps: set it before each forward pass (below 2^48; another one each time,
    where a block is applied more than once), so that every pass rounds with words of its own.
    Data-parallel ranks need words of their own too: `rank` (below 2^16) tells them apart,
    torch.distributed's where it is None and a process group is there, else 0.  Every block has its own
    words; `seed` names them instead, for words that a later run can draw again, and then blocks of one
    model need different seeds.  A captured CUDA graph replays the words of its capture.

    `products`: "bf16" for the library's products in the activations' type, "e4m3" for 8-bit floating point, which takes
    less time in large blocks, and in small ones where steps are not captured (forward and backward pass of 768 x
    3,088 over 384 tokens 79 and 99 us in a graph, 843 and 600 call after call; 4,096 x 16,384 over 8,192 tokens
    4.2 and 3.4 ms in a graph)."""

    def __init__(self, width: int, hidden: int, approximate: str = "none", eps: float = 1e-5,
                 seed: int | None = None, device=None, rank: int | None = None, products: str = "bf16"):
        super().__init__()
        self.products = products
        self._e4m3()
        self.norm_weight = nn.Parameter(torch.ones(width, device=device))
        self.norm_bias = nn.Parameter(torch.zeros(width, device=device))
        self.w1 = nn.Parameter(torch.randn(hidden, width, device=device) * width ** -0.5)
        self.b1 = nn.Parameter(torch.zeros(hidden, device=device))
        self.w2 = nn.Parameter(torch.randn(width, hidden, device=device) * hidden ** -0.5)
        self.b2 = nn.Parameter(torch.zeros(width, device=device))
        self.approximate, self.eps, self.seed, self.rank, self.step = approximate, eps, seed, rank, 0
        self._number = next(_numbers)

    def __setstate__(self, state):  # a copy, or one read back from a file
        super().__setstate__(state)
        self.__dict__.setdefault("products", "bf16")  # of a file from before it
        self._number = next(_numbers)

    def _e4m3(self):
        """Whether products are in 8-bit floating point."""
        if self.products not in ("bf16", "e4m3"):
            raise ValueError("products must be 'bf16' or 'e4m3'")
        return self.products == "e4m3"

    def words(self, layer: int):
        """(seed, step) of the random words of a layer: 0 the layer norm's checkpoint, 1 GELU's."""
        if self.seed is None:  # from the top down, where no seed is taken
            seed = (1 << 62) - 1 - self._number
        elif 0 <= self.seed < (1 << 62) - (1 << 32):
            seed = self.seed
        else:
            raise ValueError("seed must be a number below 2^62 - 2^32")
        rank = self.rank
        if rank is None:
            there = torch.distributed.is_available() and torch.distributed.is_initialized()
            rank = torch.distributed.get_rank() if there else 0
        if not (0 <= rank < 1 << 16 and 0 <= self.step < 1 << 48):
            raise ValueError("rank must be a number below 2^16 and step one below 2^48")
        return 1 << 63 | 2 * seed + layer, rank << 48 | self.step

    def forward(self, x):
        record = torch.is_grad_enabled()  # not seen within a Function's forward pass
        e4m3 = self._e4m3()
        u = _NormLinear.apply(x, self.norm_weight, self.norm_bias, self.w1, self.b1, self.eps, *self.words(0),
                              record, e4m3)
        return x + _GeluLinear.apply(u, self.w2, self.b2, self.approximate, *self.words(1), record, e4m3)
