"""8-bit activation checkpoints and the operators that write and read them (include/gq.h, the
section on activations): argument checks and marshalling over libgq.so, like _binding.

Matrices are CUDA tensors of at least two dimensions whose last one is contiguous and whose
leading ones can be viewed as one (rows may be further apart than their length); float32 or
bfloat16.  Outputs are new tensors of the same leading shape.  With `stream`, the call runs on that
stream and its new tensors belong to it.

A call on a small matrix costs more on the host than on the GPU, so the checks below read each
property once, a checkpoint is one allocation, and no context manager is entered where the
tensors' device and stream are the current ones.
"""
from __future__ import annotations

import math

import torch

from ._binding import BF16, F32, _OUT_TYPES, GQError, lib

ACT_NEAREST, ACT_RANDOM = 0, 1
GELU_ERF, GELU_TANH = 0, 1

_IN_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_FORMS = {"none": GELU_ERF, "tanh": GELU_TANH}
_empty = torch.empty


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same number without building a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(index: int, stream):
    """None if a call on tensors of device `index` can run as things stand; else the context to
    enter first: the given stream (so that new tensors belong to the stream that writes them), or
    the tensors' device."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("the stream is on %s, the tensors on cuda:%d" % (stream.device, index))
        return torch.cuda.stream(stream)
    return None if _current_device() == index else torch.cuda.device(index)


def _pitches(cols: int):
    pitch = (cols + 31) // 32 * 32
    return pitch, (pitch // 32 + 15) // 16 * 16


class Act8:
    """An 8-bit checkpoint of a rows x cols matrix: int8 codes (rows x round_up(cols, 32)) and one
    exponent byte per 32 columns (rows x round_up(ceil(cols / 32), 16)); `shape` is that of the
    tensor it was made from."""

    __slots__ = ("rows", "cols", "shape", "index", "_parts", "_data", "_pc", "_pe")

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
        self.rows, self.cols = rows, cols
        self.shape = (rows, cols) if shape is None else tuple(shape)
        self.index = codes.get_device()
        self._parts, self._data = (codes, exps), None
        self._pc, self._pe = codes.data_ptr(), exps.data_ptr()

    @property
    def codes(self) -> torch.Tensor:
        return self._views()[0]

    @property
    def exps(self) -> torch.Tensor:
        return self._views()[1]

    def _views(self):
        if self._parts is None:
            pitch, epitch = _pitches(self.cols)
            n = self.rows * pitch
            self._parts = (self._data[:n].view(torch.int8).view(self.rows, pitch),
                           self._data[n:].view(self.rows, epitch))
        return self._parts

    @property
    def nbytes(self) -> int:
        return self.rows * sum(_pitches(self.cols))


def _new_act(rows, cols, index, shape) -> Act8:
    """A checkpoint to be written: codes, then exponents, in one allocation."""
    pitch, epitch = _pitches(cols)
    a = Act8.__new__(Act8)
    a.rows, a.cols, a.shape, a.index, a._parts = rows, cols, tuple(shape), index, None
    a._data = _empty(rows * (pitch + epitch), dtype=torch.uint8, device=_device(index))
    a._pc = a._data.data_ptr()
    a._pe = a._pc + rows * pitch
    return a


_devices = {}


def _device(index: int) -> torch.device:
    d = _devices.get(index)
    if d is None:
        d = _devices[index] = torch.device("cuda", index)
    return d


def _matrix(t: torch.Tensor, what: str):
    """(type code, rows, cols, elements from one row to the next, address, device index)."""
    code = _IN_TYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (what, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    shape = t.shape
    if len(shape) != 2:
        if len(shape) < 2:
            raise ValueError("%s must have at least two dimensions" % what)
        try:
            t = t.view(math.prod(shape[:-1]), shape[-1])
        except RuntimeError:
            raise ValueError("%s: the leading dimensions cannot be viewed as one" % what) from None
        shape = t.shape
    rows, cols = shape
    ld, one = t.stride()
    if cols < 1 or (one != 1 and cols > 1):
        raise ValueError("%s: the last dimension must be contiguous and not empty" % what)
    if rows <= 1:
        ld = cols  # a single row has no next one
    elif ld < cols:
        raise ValueError("%s: rows overlap" % what)
    return code, rows, cols, ld, t.data_ptr(), t.get_device()


def _covers(act: Act8, rows: int, cols, index: int) -> None:
    if not isinstance(act, Act8):
        raise TypeError("act must be an Act8")
    if act.rows != rows or (cols is not None and act.cols != cols) or act.index != index:
        raise ValueError("the checkpoint holds %d x %d on cuda:%d" % (act.rows, act.cols, act.index))


def _vector(v, cols: int, index: int, what: str):
    """(type code, address) of a per-column vector; (None, None) for None."""
    if v is None:
        return None, None
    code = _IN_TYPES.get(v.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16" % what)
    if v.shape != (cols,) or not v.is_cuda or v.get_device() != index or not v.is_contiguous():
        raise ValueError("%s must be contiguous, %d elements, on cuda:%d" % (what, cols, index))
    return code, v.data_ptr()


def _floats(v, n: int, index: int, what: str) -> int:
    if v.dtype != torch.float32 or v.shape != (n,) or not v.is_cuda or v.get_device() != index \
            or not v.is_contiguous():
        raise ValueError("%s must be contiguous float32, %d elements, on cuda:%d" % (what, n, index))
    return v.data_ptr()


def _rounding(seed, step):
    if seed is None:
        return ACT_NEAREST, 0, 0
    if not 0 <= seed < 1 << 64 or not 0 <= step < 1 << 64:
        raise ValueError("seed and step must be unsigned 64-bit numbers")
    return ACT_RANDOM, seed, step


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
    code, rows, outs, ld, p, _ = _matrix(dy, "dy")
    return lib().gq_linear_wgrad_workspace_bytes(p, code, rows, outs, ld, cols)


def _workspace(ws, nbytes: int, index: int):
    """The workspace tensor, its address and size in bytes."""
    if ws is None:
        ws = _empty(nbytes, dtype=torch.uint8, device=_device(index))
        return ws, ws.data_ptr(), nbytes
    if not ws.is_cuda or ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on cuda:%d" % index)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _like(t: torch.Tensor) -> torch.Tensor:
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def gq_act_quantize(x, seed=None, step=0, stream=None) -> Act8:
    """8-bit checkpoint of x: rounded to nearest (seed None), or at random without bias."""
    code, rows, cols, ld, p, index = _matrix(x, "x")
    rounding, seed, step = _rounding(seed, step)
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_act_quantize(x, seed if rounding else None, step)
    act = _new_act(rows, cols, index, x.shape)
    rc = lib().gq_act_quantize(p, code, rows, cols, ld, rounding, seed, step, act._pc, act._pe,
                               _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_act_quantize")
    return act


def gq_act_dequantize(act, out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of a checkpoint (float32, bfloat16 or float16), in `out` or a new tensor."""
    if not isinstance(act, Act8):
        raise TypeError("act must be an Act8")
    index = act.index
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_act_dequantize(act, out, out_dtype)
    rows, cols = act.rows, act.cols
    ld = cols
    if out is None:
        out = _empty(act.shape, dtype=out_dtype, device=_device(index))
    code = _OUT_TYPES.get(out.dtype)
    if code is None:
        raise TypeError("values are float32, bfloat16 or float16")
    if not out.is_contiguous() or out.numel() != rows * cols or out.shape[-1] != cols:
        if out.numel() != rows * cols or out.dim() != 2 or out.shape[1] != cols or \
                (out.stride(1) != 1 and cols > 1) or (rows > 1 and out.stride(0) < cols):
            raise ValueError("out must hold %d x %d, its rows contiguous" % (rows, cols))
        ld = out.stride(0) if rows > 1 else cols
    if not out.is_cuda or out.get_device() != index:
        raise ValueError("out must be on cuda:%d" % index)
    rc = lib().gq_act_dequantize(act._pc, act._pe, rows, cols, out.data_ptr(), code, ld,
                                 _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_act_dequantize")
    return out


def gq_layernorm_forward(x, weight=None, bias=None, eps=1e-5, checkpoint=True, seed=None, step=0,
                         stream=None):
    """(y, mean, rstd, act): layer norm of every row of x; act is the 8-bit checkpoint of the
    normalised rows (None with checkpoint=False)."""
    code, rows, cols, ld, p, index = _matrix(x, "x")
    wtype, pw = _vector(weight, cols, index, "weight")
    btype, pb = _vector(bias, cols, index, "bias")
    if wtype != btype and wtype is not None and btype is not None:
        raise TypeError("weight and bias must be of one type")
    rounding, seed, step = _rounding(seed, step)
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_layernorm_forward(x, weight, bias, eps, checkpoint, seed if rounding else None,
                                        step)
    y = _like(x)
    mean = _empty(rows, dtype=torch.float32, device=_device(index))
    rstd = _empty(rows, dtype=torch.float32, device=_device(index))
    act = pc = pe = None
    if checkpoint:
        act = _new_act(rows, cols, index, x.shape)
        pc, pe = act._pc, act._pe
    rc = lib().gq_layernorm_forward(
        p, code, rows, cols, ld, pw, pb, wtype or btype or F32, eps, y.data_ptr(), cols, mean.data_ptr(),
        rstd.data_ptr(), rounding, seed, step, pc, pe, _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_layernorm_forward")
    return y, mean, rstd, act


def gq_layernorm_backward(dy, weight, rstd, act=None, x=None, mean=None, grad_dtype=torch.float32,
                          ws=None, stream=None):
    """(dx, dweight, dbias) from the checkpoint of the normalised rows, or from x and mean;
    dweight and dbias are of grad_dtype (float32 or bfloat16)."""
    code, rows, cols, ld, p, index = _matrix(dy, "dy")
    wtype, pw = _vector(weight, cols, index, "weight")
    gtype = _IN_TYPES.get(grad_dtype)
    if gtype is None:
        raise TypeError("grad_dtype must be float32 or bfloat16")
    if (act is None) == (x is None) or (x is None) != (mean is None):
        raise ValueError("give either act, or x and mean")
    pr = _floats(rstd, rows, index, "rstd")
    pc = pe = px = pm = None
    ldx = 0
    if act is not None:
        _covers(act, rows, cols, index)
        pc, pe = act._pc, act._pe
    else:
        xcode, xrows, xcols, ldx, px, xindex = _matrix(x, "x")
        if (xcode, xrows, xcols, xindex) != (code, rows, cols, index):
            raise ValueError("x must match dy in shape, type and device")
        pm = _floats(mean, rows, index, "mean")
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_layernorm_backward(dy, weight, rstd, act, x, mean, grad_dtype, ws)
    L = lib()
    ws, pws, nbytes = _workspace(ws, L.gq_layernorm_workspace_bytes(rows, cols) if ws is None else 0,
                                 index)
    dx = _like(dy)
    dw = _empty(cols, dtype=grad_dtype, device=_device(index))
    db = _empty(cols, dtype=grad_dtype, device=_device(index))
    rc = L.gq_layernorm_backward(
        p, code, rows, cols, ld, pw, F32 if wtype is None else wtype, pr, pc, pe, px, ldx, pm,
        dx.data_ptr(), cols, dw.data_ptr(), db.data_ptr(), gtype, pws, nbytes, _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_layernorm_backward")
    return dx, dw, db


def gq_gelu_forward(u, approximate="none", checkpoint=True, seed=None, step=0, stream=None):
    """(h, act): h = gelu(u) (approximate as torch's: "none" or "tanh") and the 8-bit checkpoint of
    u (None with checkpoint=False)."""
    code, rows, cols, ld, p, index = _matrix(u, "u")
    form = _form(approximate)
    rounding, seed, step = _rounding(seed, step)
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_gelu_forward(u, approximate, checkpoint, seed if rounding else None, step)
    h = _like(u)
    act = pc = pe = None
    if checkpoint:
        act = _new_act(rows, cols, index, u.shape)
        pc, pe = act._pc, act._pe
    rc = lib().gq_gelu_forward(p, code, rows, cols, ld, form, h.data_ptr(), cols, rounding, seed, step,
                               pc, pe, _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_gelu_forward")
    return h, act


def gq_gelu_backward(dh, act, approximate="none", need_output=False, stream=None):
    """du = dh gelu'(u) with u from its checkpoint; with need_output (du, gelu(u))."""
    code, rows, cols, ld, p, index = _matrix(dh, "dh")
    form = _form(approximate)
    _covers(act, rows, cols, index)
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_gelu_backward(dh, act, approximate, need_output)
    du = _like(dh)
    h = _like(dh) if need_output else None
    rc = lib().gq_gelu_backward(p, code, rows, cols, ld, act._pc, act._pe, form, du.data_ptr(), cols,
                                h.data_ptr() if need_output else None, cols, _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_gelu_backward")
    return (du, h) if need_output else du


def gq_linear_wgrad(dy, act, scale=None, shift=None, out_dtype=torch.float32, need_bias=True, ws=None,
                    stream=None):
    """(dw, dbias) of a linear layer from the gradient of its output (rows x outs) and the
    checkpoint of its input, or of that input's value before a per-column scale and shift (float32;
    a layer norm's weight and bias).  dw: outs x cols of out_dtype; dbias: float32, None without
    need_bias."""
    code, rows, outs, ld, p, index = _matrix(dy, "dy")
    _covers(act, rows, None, index)
    cols = act.cols
    otype = _IN_TYPES.get(out_dtype)
    if otype is None:
        raise TypeError("out_dtype must be float32 or bfloat16")
    stype, ps = _vector(scale, cols, index, "scale")
    htype, ph = _vector(shift, cols, index, "shift")
    if stype or htype:  # a type other than F32
        raise TypeError("scale and shift must be float32")
    there = _elsewhere(index, stream)
    if there is not None:
        with there:
            return gq_linear_wgrad(dy, act, scale, shift, out_dtype, need_bias, ws)
    L = lib()
    ws, pws, nbytes = _workspace(
        ws, L.gq_linear_wgrad_workspace_bytes(p, code, rows, outs, ld, cols) if ws is None else 0, index)
    dw = _empty((outs, cols), dtype=out_dtype, device=_device(index))
    db = _empty(outs, dtype=torch.float32, device=_device(index)) if need_bias else None
    rc = L.gq_linear_wgrad(p, code, rows, outs, ld, act._pc, act._pe, cols, ps, ph, dw.data_ptr(), otype,
                           cols, db.data_ptr() if need_bias else None, pws, nbytes, _raw_stream(index))
    if rc:
        raise GQError(rc, "gq_linear_wgrad")
    return dw, db
