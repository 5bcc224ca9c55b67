"""8-bit activation checkpoints and the operators that write and read them (include/gq.h, the
section on activations): argument checks and marshalling over libgq.so, like _binding.

Matrices are CUDA tensors of at least two dimensions whose last one is contiguous and whose
leading ones can be viewed as one (rows may be further apart than their length); float32 or
bfloat16.  Outputs are new tensors of the same leading shape.  With `stream`, the call runs on that
stream and its new tensors belong to it.  Like every call of this package they are not recorded by
autograd: outputs do not require gradients, whatever the inputs do (act8_layers has autograd functions
over them).

The checks, the allocations and the calls are in csrc/gq_native.cpp: on a small matrix they would take
longer in Python than the kernels on the GPU.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import _build
from ._binding import _OUT_TYPES, GQError, lib

ACT_NEAREST, ACT_RANDOM = 0, 1
GELU_ERF, GELU_TANH = 0, 1

_FORMS = {"none": GELU_ERF, "tanh": GELU_TANH}
_FUNCTIONS = ("gq_act_quantize", "gq_act_dequantize", "gq_layernorm_forward",
              "gq_layernorm_workspace_bytes", "gq_layernorm_backward", "gq_gelu_forward",
              "gq_gelu_backward", "gq_linear_wgrad_workspace_bytes", "gq_linear_wgrad_plan",
              "gq_linear_wgrad")


def load_native():
    """The extension module, calling the loaded libgq.so; fails loudly if either is not built."""
    path = _build.native_path()
    if not os.path.exists(path):
        raise ImportError("%s is not built: run `python -c \"import __graft_entry__ as g; g.build()\"` "
                          "first; there is no fallback path" % os.path.basename(path))
    loader = importlib.machinery.ExtensionFileLoader("gq_native", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("gq_native", loader))
    loader.exec_module(module)
    module.bind(GQError, *[ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value for f in _FUNCTIONS])
    return module


class _Native:
    """The extension module, loaded when an operator is first called."""

    def __getattr__(self, name):
        global _native
        _native = load_native()
        return getattr(_native, name)


_native = _Native()


def _on(stream, call, *args):
    """call(*args) on a stream, whose device becomes current too."""
    with torch.cuda.stream(stream):
        return call(*args)


def _pitches(cols: int):
    pitch = (cols + 31) // 32 * 32
    return pitch, (pitch // 32 + 15) // 16 * 16


class Act8:
    """An 8-bit checkpoint of a rows x cols matrix: int8 codes (rows x round_up(cols, 32)) and one
    exponent byte per 32 columns (rows x round_up(ceil(cols / 32), 16)); `shape` is that of the
    tensor it was made from."""

    __slots__ = ("shape", "_cols", "_codes", "_exps")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, cols: int, shape=None):
        rows = codes.shape[0] if codes.dim() == 2 else -1
        pitch, epitch = _pitches(cols)
        if cols < 1 or rows < 0 or codes.shape[1] != pitch or exps.shape != (rows, epitch):
            raise ValueError("a checkpoint of %d columns has codes of rows x %d and exponents of "
                             "rows x %d, got %s and %s" % (cols, pitch, epitch, tuple(codes.shape),
                                                           tuple(exps.shape)))
        if codes.dtype != torch.int8 or exps.dtype != torch.uint8:
            raise TypeError("codes must be int8 and exponents uint8")
        if not codes.is_contiguous() or not exps.is_contiguous():
            raise ValueError("codes and exponents must be contiguous")
        if not codes.is_cuda or codes.get_device() != exps.get_device():
            raise ValueError("codes and exponents must be on one CUDA device")
        self.shape = (rows, cols) if shape is None else tuple(shape)
        self._cols, self._codes, self._exps = cols, codes, exps

    @classmethod
    def of_data(cls, data: torch.Tensor, cols: int, shape=None) -> "Act8":
        """The checkpoint whose `data` this is: for code that keeps tensors and not objects, as autograd
        functions do."""
        self = cls.__new__(cls)
        self.shape = (data.shape[0], cols) if shape is None else tuple(shape)
        self._cols, self._codes, self._exps = cols, data, None
        return self

    @property
    def data(self) -> torch.Tensor:
        """What a call has written, one tensor of bytes: the codes of all rows, then the exponents (None
        for a checkpoint made of two tensors)."""
        return self._codes if self._exps is None else None

    @property
    def rows(self) -> int:
        return self._codes.shape[0]

    @property
    def cols(self) -> int:
        return self._cols

    @property
    def codes(self) -> torch.Tensor:
        if self._exps is not None:
            return self._codes
        pitch = _pitches(self._cols)[0]
        return self._codes.view(-1)[:self.rows * pitch].view(torch.int8).view(self.rows, pitch)

    @property
    def exps(self) -> torch.Tensor:
        if self._exps is not None:
            return self._exps
        pitch, epitch = _pitches(self._cols)
        return self._codes.view(-1)[self.rows * pitch:].view(self.rows, epitch)

    @property
    def nbytes(self) -> int:
        return self.rows * sum(_pitches(self._cols))


def _place_of(act):
    """What the calls take of a checkpoint: its tensors, whose addresses they read themselves, so that a
    copy, or new storage, is never read at an old address."""
    if type(act) is not Act8:
        raise TypeError("act must be an Act8")
    return act._codes, act._exps, act._cols


def _form(approximate: str) -> int:
    form = _FORMS.get(approximate)
    if form is None:
        raise ValueError("approximate must be 'none' or 'tanh'")
    return form


def gq_act_exp_pitch(cols: int) -> int:
    return lib().gq_act_exp_pitch(cols)


def gq_layernorm_workspace_bytes(rows: int, cols: int) -> int:
    return lib().gq_layernorm_workspace_bytes(rows, cols)


def gq_linear_wgrad_workspace_bytes(dy: torch.Tensor, cols: int) -> int:
    return _native.linear_wgrad_workspace_bytes(dy, cols)


_PLAN = ("tile_outs", "tile_cols", "steps", "shares", "own", "left", "longest", "chain")


def gq_linear_wgrad_plan(dy: torch.Tensor, cols: int) -> dict:
    """How gq_linear_wgrad divides its work for this dy and a checkpoint of `cols` columns (include/gq.h)."""
    return dict(zip(_PLAN, _native.linear_wgrad_plan(dy, cols)))


def gq_act_quantize(x, seed=None, step=0, stream=None) -> Act8:
    """8-bit checkpoint of x: rounded to nearest (seed None), or at random without bias."""
    if stream is not None:
        return _on(stream, gq_act_quantize, x, seed, step)
    return Act8.of_data(_native.act_quantize(x, seed, step), x.shape[-1], x.shape)


def gq_act_dequantize(act, out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of a checkpoint (float32, bfloat16 or float16), in `out` or a new tensor."""
    if stream is not None:
        return _on(stream, gq_act_dequantize, act, out, out_dtype)
    return _native.act_dequantize(*_place_of(act), act.shape, out, _OUT_TYPES.get(out_dtype, -1))


def gq_layernorm_forward(x, weight=None, bias=None, eps=1e-5, checkpoint=True, seed=None, step=0,
                         stream=None):
    """(y, mean, rstd, act): layer norm of every row of x; act is the 8-bit checkpoint of the
    normalised rows (None with checkpoint=False)."""
    if stream is not None:
        return _on(stream, gq_layernorm_forward, x, weight, bias, eps, checkpoint, seed, step)
    y, mean, rstd, data = _native.layernorm_forward(x, weight, bias, eps, checkpoint, seed, step)
    return y, mean, rstd, None if data is None else Act8.of_data(data, x.shape[-1], x.shape)


def gq_layernorm_backward(dy, weight, rstd, act=None, x=None, mean=None, grad_dtype=torch.float32,
                          ws=None, stream=None):
    """(dx, dweight, dbias) from the checkpoint of the normalised rows, or from x and mean;
    dweight and dbias are of grad_dtype (float32 or bfloat16)."""
    if stream is not None:
        return _on(stream, gq_layernorm_backward, dy, weight, rstd, act, x, mean, grad_dtype, ws)
    at = (None,) * 3 if act is None else _place_of(act)
    return _native.layernorm_backward(dy, weight, rstd, *at, x, mean, _OUT_TYPES.get(grad_dtype, -1), ws)


def gq_gelu_forward(u, approximate="none", checkpoint=True, seed=None, step=0, stream=None):
    """(h, act): h = gelu(u) (approximate as torch's: "none" or "tanh") and the 8-bit checkpoint of
    u (None with checkpoint=False)."""
    if stream is not None:
        return _on(stream, gq_gelu_forward, u, approximate, checkpoint, seed, step)
    h, data = _native.gelu_forward(u, _form(approximate), checkpoint, seed, step)
    return h, None if data is None else Act8.of_data(data, u.shape[-1], u.shape)


def gq_gelu_backward(dh, act, approximate="none", need_output=False, stream=None):
    """du = dh gelu'(u) with u from its checkpoint; with need_output (du, gelu(u))."""
    if stream is not None:
        return _on(stream, gq_gelu_backward, dh, act, approximate, need_output)
    return _native.gelu_backward(dh, *_place_of(act), _form(approximate), need_output)


def gq_linear_wgrad(dy, act, scale=None, shift=None, out_dtype=torch.float32, need_bias=True, ws=None,
                    stream=None):
    """(dw, dbias) of a linear layer from the gradient of its output (rows x outs) and the
    checkpoint of its input, or of that input's value before a per-column scale and shift (float32;
    a layer norm's weight and bias).  dw: outs x cols of out_dtype; dbias: float32, None without
    need_bias."""
    if stream is not None:
        return _on(stream, gq_linear_wgrad, dy, act, scale, shift, out_dtype, need_bias, ws)
    return _native.linear_wgrad(dy, *_place_of(act), scale, shift, _OUT_TYPES.get(out_dtype, -1), need_bias,
                                ws)
