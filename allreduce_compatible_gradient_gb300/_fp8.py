"""Matrices in 8-bit floating point and the products of a linear layer on them (include/gq.h, the section
on 8-bit floating point): argument checks and marshalling over libgq.so, like _activations, with the same
rules for matrices, streams and autograd.
"""
from __future__ import annotations

import math

import torch

from . import _activations as _acts
from ._activations import _on
from ._binding import _OUT_TYPES, lib


def gq_fp8_code_pitch(cols: int) -> int:
    return lib().gq_fp8_code_pitch(cols)


def gq_fp8_exp_bytes(rows: int, cols: int) -> int:
    return lib().gq_fp8_exp_bytes(rows, cols)


def gq_fp8_linear_workspace_bytes(rows: int, depth: int, outs: int) -> int:
    return lib().gq_fp8_linear_workspace_bytes(rows, depth, outs)


def _up(v, m):
    return (v + m - 1) // m * m


def _exp_shape(rows, cols):
    return (rows + 127) // 128, (cols + 511) // 512, 32, 4, 4


class Fp8:
    """A rows x cols matrix in 8-bit floating point: e4m3 codes (rows x round_up(cols, 16) bytes) and an
    exponent byte per 128 columns of each row, as the tensor cores read them ([ceil(rows / 128)]
    [ceil(cols / 512)][32][4][4]).  exps_t: those of the transposed matrix, where 128 x 128 elements share
    one (`tiles`).  `shape` is that of the tensor it was made from."""

    __slots__ = ("shape", "_rows", "_cols", "_tiles", "_codes", "_exps", "_exps_t")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, cols: int, exps_t: torch.Tensor | None = None,
                 shape=None):
        rows, pitch = codes.shape if codes.dim() == 2 else (-1, 0)
        if cols < 1 or rows < 0 or pitch != (cols + 15) // 16 * 16 or exps.shape != _exp_shape(rows, cols):
            raise ValueError("a matrix of %d columns has codes of rows x %d and exponents %s, got %s and %s"
                             % (cols, _up(cols, 16), _exp_shape(max(rows, 0), cols), tuple(codes.shape),
                                tuple(exps.shape)))
        if exps_t is not None and exps_t.shape != _exp_shape(cols, rows):
            raise ValueError("the transposed matrix has exponents %s, got %s"
                             % (_exp_shape(cols, rows), tuple(exps_t.shape)))
        if (codes.dtype is not torch.uint8 and codes.dtype is not torch.float8_e4m3fn
                or exps.dtype is not torch.uint8 or exps_t is not None and exps_t.dtype is not torch.uint8):
            raise TypeError("codes must be uint8 or float8_e4m3fn and exponents uint8")
        # (that all of it is contiguous, and on one device, is checked by every call)
        self.shape = (rows, cols) if shape is None else tuple(shape)
        self._rows, self._cols, self._tiles = rows, cols, exps_t is not None
        self._codes, self._exps, self._exps_t = codes, exps, exps_t

    @classmethod
    def of_data(cls, data: torch.Tensor, rows: int, cols: int, tiles: bool = False, shape=None) -> "Fp8":
        """The matrix whose `data` this is: for code that keeps tensors and not objects, as autograd functions
        do."""
        self = cls.__new__(cls)
        self.shape = (rows, cols) if shape is None else tuple(shape)
        self._rows, self._cols, self._tiles = rows, cols, tiles
        self._codes, self._exps, self._exps_t = data, None, None
        return self

    @property
    def data(self) -> torch.Tensor:
        """What a call has written, one tensor of bytes: codes, exponents, and (tiles) those of the transposed
        matrix (None for a matrix made of several tensors)."""
        return self._codes if self._exps is None else None

    @property
    def rows(self) -> int:
        return self._rows

    @property
    def cols(self) -> int:
        return self._cols

    @property
    def tiles(self) -> bool:
        """Whether 128 x 128 elements share an exponent and those of the transposed matrix are there."""
        return self._tiles

    def _part(self, k):
        have = (self._codes, self._exps, self._exps_t)
        if self._exps is not None:
            return have[k]
        pitch = _up(self._cols, 16)
        shapes = ((self._rows, pitch), _exp_shape(self._rows, self._cols), _exp_shape(self._cols, self._rows))
        if k == 2 and not self._tiles:
            return None
        sizes = [math.prod(v) for v in shapes]
        at = sum(sizes[:k])
        return self._codes[at:at + sizes[k]].view(shapes[k])

    @property
    def codes(self) -> torch.Tensor:
        return self._part(0).view(torch.float8_e4m3fn)

    @property
    def exps(self) -> torch.Tensor:
        return self._part(1)

    @property
    def exps_t(self) -> torch.Tensor | None:
        return self._part(2)

    @property
    def blocks(self) -> torch.Tensor:
        """The exponent bytes as a matrix: rows x ceil(cols / 128)."""
        e = self.exps.permute(0, 3, 2, 1, 4)
        return e.reshape(e.shape[0] * 128, -1)[:self._rows, :(self._cols + 127) // 128]

    @property
    def nbytes(self) -> int:
        return sum(t.numel() for t in (self._codes, self._exps, self._exps_t) if t is not None)


_NONE = (None,) * 7


def _place_of(f, what):
    """What the calls take of a matrix: its tensors, whose addresses they read themselves."""
    if type(f) is not Fp8:
        raise TypeError("%s must be an Fp8" % what)
    return f._codes, f._exps, f._exps_t, f._rows, f._cols, f._tiles


def _tokens(x, what):
    return (x, *_NONE) if isinstance(x, torch.Tensor) else (None, *_place_of(x, what), x.shape)


def _out(x, out_dtype):
    if out_dtype is None:
        out_dtype = x.dtype if isinstance(x, torch.Tensor) else torch.bfloat16
    return _OUT_TYPES.get(out_dtype, -1)


def gq_fp8_quantize(x, tiles=False, stream=None) -> Fp8:
    """x (float32 or bfloat16) in 8-bit floating point, with an exponent per 128 columns of a row (activations,
    gradients), or per 128 x 128 elements (tiles: weights)."""
    if stream is not None:
        return _on(stream, gq_fp8_quantize, x, tiles)
    data = _acts._native.fp8_quantize(x, tiles)
    cols = x.shape[-1]
    return Fp8.of_data(data, x.numel() // cols, cols, bool(tiles), x.shape)


def gq_fp8_dequantize(f, out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of a matrix (float32, bfloat16 or float16), in `out` or a new tensor."""
    if stream is not None:
        return _on(stream, gq_fp8_dequantize, f, out, out_dtype)
    return _acts._native.fp8_dequantize(*_place_of(f, "f"), f.shape, out, _OUT_TYPES.get(out_dtype, -1))


def gq_fp8_linear(x, weight, bias=None, out_dtype=None, stream=None) -> torch.Tensor:
    """x weight^T + bias on operands in 8-bit floating point.  x: a tensor (float32 or bfloat16), put into it
    by the call, or an Fp8 (tiles=False); weight: an Fp8 of outs x cols; bias: float32.  out_dtype: float32 or
    bfloat16, x's where it is None (bfloat16 for an Fp8)."""
    if stream is not None:
        return _on(stream, gq_fp8_linear, x, weight, bias, out_dtype)
    return _acts._native.fp8_linear(*_tokens(x, "x"), *_place_of(weight, "weight"), bias, _out(x, out_dtype))


def gq_fp8_linear_dgrad(dy, weight, out_dtype=None, stream=None) -> torch.Tensor:
    """dy weight, the gradient of gq_fp8_linear's x.  dy as x there; weight: an Fp8 made with tiles=True."""
    if stream is not None:
        return _on(stream, gq_fp8_linear_dgrad, dy, weight, out_dtype)
    return _acts._native.fp8_linear_dgrad(*_tokens(dy, "dy"), *_place_of(weight, "weight"), _out(dy, out_dtype))
