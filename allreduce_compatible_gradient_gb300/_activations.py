"""8-bit activation checkpoints and the operators that write and read them (include/gq.h, the
section on activations): argument checks and marshalling over libgq.so, like _binding.

Matrices are CUDA tensors of at least two dimensions whose last one is contiguous and whose
leading ones can be viewed as one (rows may be further apart than their length); float32 or
bfloat16.  Outputs are new tensors of the same leading shape.  With `stream`, the call runs on that
stream and its new tensors belong to it.
"""
from __future__ import annotations

import contextlib
import math

import torch

from ._binding import BF16, F32, _OUT_TYPES, _check, lib

ACT_NEAREST, ACT_RANDOM = 0, 1
GELU_ERF, GELU_TANH = 0, 1

_IN_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_FORMS = {"none": GELU_ERF, "tanh": GELU_TANH}
_HERE = contextlib.nullcontext()


class Act8:
    """An 8-bit checkpoint of a rows x cols matrix: int8 codes (rows x round_up(cols, 32)) and one
    exponent byte per 32 columns (rows x round_up(ceil(cols / 32), 16)); `shape` is that of the
    tensor it was made from."""

    __slots__ = ("codes", "exps", "cols", "shape")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, cols: int, shape=None):
        rows = codes.shape[0] if codes.dim() == 2 else -1
        pitch = (cols + 31) // 32 * 32
        epitch = (pitch // 32 + 15) // 16 * 16
        if cols < 1 or codes.dim() != 2 or codes.shape[1] != pitch or \
                exps.shape != (rows, epitch):
            raise ValueError("a checkpoint of %d columns has codes of rows x %d and exponents of "
                             "rows x %d, got %s and %s" % (cols, pitch, epitch, tuple(codes.shape),
                                                           tuple(exps.shape)))
        if codes.dtype != torch.int8 or exps.dtype != torch.uint8:
            raise TypeError("codes must be int8 and exponents uint8")
        if not codes.is_contiguous() or not exps.is_contiguous():
            raise ValueError("codes and exponents must be contiguous")
        if codes.device != exps.device:
            raise ValueError("codes and exponents must be on one device")
        self.codes, self.exps, self.cols = codes, exps, cols
        self.shape = (rows, cols) if shape is None else tuple(shape)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.exps.numel()


def _matrix(t: torch.Tensor, what: str) -> torch.Tensor:
    """t as a two-dimensional view."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if t.dtype not in _IN_TYPES:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (what, t.dtype))
    if t.dim() != 2:
        if t.dim() < 2:
            raise ValueError("%s must have at least two dimensions" % what)
        try:
            t = t.view(math.prod(t.shape[:-1]), t.shape[-1])
        except RuntimeError:
            raise ValueError("%s: the leading dimensions cannot be viewed as one" % what) from None
    if t.shape[1] < 1 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("%s: the last dimension must be contiguous and not empty" % what)
    return t


def _ld(t: torch.Tensor) -> int:
    """Elements from one row to the next; a single row has no next one."""
    ld = t.stride(0)
    if t.shape[0] <= 1:
        return t.shape[1]
    if ld < t.shape[1]:
        raise ValueError("rows overlap")
    return ld


def _same(t: torch.Tensor, like: torch.Tensor, what: str) -> torch.Tensor:
    t = _matrix(t, what)
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError("%s must match in shape, type and device" % what)
    return t


def _covers(act: Act8, rows: int, cols, device) -> None:
    if not isinstance(act, Act8):
        raise TypeError("act must be an Act8")
    if act.rows != rows or (cols is not None and act.cols != cols) or act.codes.device != device:
        raise ValueError("the checkpoint holds %d x %d on %s" % (act.rows, act.cols,
                                                                 act.codes.device))


def _vectors(cols: int, device, *vectors):
    """Type code of the per-column vectors that are given (all of one type)."""
    code = None
    for v in vectors:
        if v is None:
            continue
        if v.dtype not in _IN_TYPES:
            raise TypeError("per-column vectors must be float32 or bfloat16")
        if v.shape != (cols,) or v.device != device or not v.is_contiguous():
            raise ValueError("per-column vectors must be contiguous, %d elements, on %s"
                             % (cols, device))
        if code is not None and _IN_TYPES[v.dtype] != code:
            raise TypeError("weight and bias must be of one type")
        code = _IN_TYPES[v.dtype]
    return F32 if code is None else code


def _place(device, stream):
    """The context in which to allocate and launch: the tensors' device, and `stream` if given (so
    that new tensors belong to the stream that writes them)."""
    if stream is not None:
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _rounding(seed):
    if seed is None:
        return ACT_NEAREST, 0
    if not 0 <= seed < 1 << 64:
        raise ValueError("seed must be an unsigned 64-bit number")
    return ACT_RANDOM, seed


def _step(step):
    if not 0 <= step < 1 << 64:
        raise ValueError("step must be an unsigned 64-bit number")
    return step


def _new_act(rows, cols, device, shape) -> Act8:
    pitch = (cols + 31) // 32 * 32
    a = Act8.__new__(Act8)
    a.codes = torch.empty((rows, pitch), dtype=torch.int8, device=device)
    a.exps = torch.empty((rows, (pitch // 32 + 15) // 16 * 16), dtype=torch.uint8, device=device)
    a.cols, a.shape = cols, tuple(shape)
    return a


def _form(approximate: str) -> int:
    if approximate not in _FORMS:
        raise ValueError("approximate must be 'none' or 'tanh'")
    return _FORMS[approximate]


def gq_act_exp_pitch(cols: int) -> int:
    return lib().gq_act_exp_pitch(cols)


def gq_layernorm_workspace_bytes(rows: int, cols: int) -> int:
    return lib().gq_layernorm_workspace_bytes(rows, cols)


def gq_linear_wgrad_workspace_bytes(dy: torch.Tensor, cols: int) -> int:
    d = _matrix(dy, "dy")
    return lib().gq_linear_wgrad_workspace_bytes(d.data_ptr(), _IN_TYPES[d.dtype], d.shape[0],
                                                 d.shape[1], _ld(d), cols)


def _workspace(ws, nbytes: int, device) -> torch.Tensor:
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on %s" % device)
    return ws


def gq_act_quantize(x, seed=None, step=0, stream=None) -> Act8:
    """8-bit checkpoint of x: rounded to nearest (seed None), or at random without bias."""
    m = _matrix(x, "x")
    rounding, key = _rounding(seed)
    rows, cols = m.shape
    with _place(m.device, stream):
        act = _new_act(rows, cols, m.device, x.shape)
        _check(lib().gq_act_quantize(m.data_ptr(), _IN_TYPES[m.dtype], rows, cols, _ld(m), rounding,
                                     key, _step(step), act.codes.data_ptr(), act.exps.data_ptr(),
                                     _raw_stream(m.device)), "gq_act_quantize")
    return act


def gq_act_dequantize(act, out=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of a checkpoint (float32, bfloat16 or float16), in `out` or a new tensor."""
    if not isinstance(act, Act8):
        raise TypeError("act must be an Act8")
    device = act.codes.device
    if device.type != "cuda":
        raise ValueError("the checkpoint must be on a CUDA device")
    with _place(device, stream):
        if out is None:
            out = torch.empty(act.shape, dtype=out_dtype, device=device)
        if out.dtype not in _OUT_TYPES:
            raise TypeError("values are float32, bfloat16 or float16")
        if out.numel() != act.rows * act.cols or out.shape[-1] != act.cols or out.device != device:
            raise ValueError("out must hold %d x %d on %s" % (act.rows, act.cols, device))
        o = out if out.dim() == 2 else out.view(act.rows, act.cols)
        if o.stride(1) != 1 and act.cols > 1:
            raise ValueError("out: the last dimension must be contiguous")
        _check(lib().gq_act_dequantize(act.codes.data_ptr(), act.exps.data_ptr(), act.rows, act.cols,
                                       o.data_ptr(), _OUT_TYPES[o.dtype], _ld(o),
                                       _raw_stream(device)), "gq_act_dequantize")
    return out


def gq_layernorm_forward(x, weight=None, bias=None, eps=1e-5, checkpoint=True, seed=None, step=0,
                         stream=None):
    """(y, mean, rstd, act): layer norm of every row of x; act is the 8-bit checkpoint of the
    normalised rows (None with checkpoint=False)."""
    m = _matrix(x, "x")
    rows, cols = m.shape
    device = m.device
    wtype = _vectors(cols, device, weight, bias)
    rounding, key = _rounding(seed)
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    with _place(device, stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=device)
        stats = torch.empty((2, rows), dtype=torch.float32, device=device)
        act = _new_act(rows, cols, device, x.shape) if checkpoint else None
        _check(lib().gq_layernorm_forward(
            m.data_ptr(), _IN_TYPES[m.dtype], rows, cols, _ld(m),
            None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(),
            wtype, eps, y.data_ptr(), cols, stats.data_ptr(), stats.data_ptr() + 4 * rows, rounding, key,
            _step(step), act.codes.data_ptr() if checkpoint else None,
            act.exps.data_ptr() if checkpoint else None, _raw_stream(device)), "gq_layernorm_forward")
    return y, stats[0], stats[1], act


def gq_layernorm_backward(dy, weight, rstd, act=None, x=None, mean=None, grad_dtype=torch.float32,
                          ws=None, stream=None):
    """(dx, dweight, dbias) from the checkpoint of the normalised rows, or from x and mean;
    dweight and dbias are of grad_dtype (float32 or bfloat16)."""
    d = _matrix(dy, "dy")
    rows, cols = d.shape
    device = d.device
    wtype = _vectors(cols, device, weight)
    if grad_dtype not in _IN_TYPES:
        raise TypeError("grad_dtype must be float32 or bfloat16")
    if (act is None) == (x is None) or (x is None) != (mean is None):
        raise ValueError("give either act, or x and mean")
    for v in (rstd, mean):
        if v is not None and (v.dtype != torch.float32 or v.shape != (rows,) or v.device != device
                              or not v.is_contiguous()):
            raise ValueError("rstd and mean must be contiguous float32, %d elements" % rows)
    if act is not None:
        _covers(act, rows, cols, device)
    else:
        x = _same(x, d, "x")
    with _place(device, stream):
        ws = _workspace(ws, lib().gq_layernorm_workspace_bytes(rows, cols), device)
        dx = torch.empty(dy.shape, dtype=dy.dtype, device=device)
        dwb = torch.empty((2, cols), dtype=grad_dtype, device=device)
        dw, db = dwb[0], dwb[1]
        _check(lib().gq_layernorm_backward(
            d.data_ptr(), _IN_TYPES[d.dtype], rows, cols, _ld(d),
            None if weight is None else weight.data_ptr(), wtype, rstd.data_ptr(),
            None if act is None else act.codes.data_ptr(),
            None if act is None else act.exps.data_ptr(), None if x is None else x.data_ptr(),
            0 if x is None else _ld(x), None if mean is None else mean.data_ptr(), dx.data_ptr(), cols,
            dw.data_ptr(), db.data_ptr(), _IN_TYPES[grad_dtype], ws.data_ptr(),
            ws.numel() * ws.element_size(), _raw_stream(device)), "gq_layernorm_backward")
    return dx, dw, db


def gq_gelu_forward(u, approximate="none", checkpoint=True, seed=None, step=0, stream=None):
    """(h, act): h = gelu(u) (approximate as torch's: "none" or "tanh") and the 8-bit checkpoint of
    u (None with checkpoint=False)."""
    m = _matrix(u, "u")
    rows, cols = m.shape
    form = _form(approximate)
    rounding, key = _rounding(seed)
    with _place(m.device, stream):
        h = torch.empty(u.shape, dtype=u.dtype, device=m.device)
        act = _new_act(rows, cols, m.device, u.shape) if checkpoint else None
        _check(lib().gq_gelu_forward(m.data_ptr(), _IN_TYPES[m.dtype], rows, cols, _ld(m), form,
                                     h.data_ptr(), cols, rounding, key, _step(step),
                                     act.codes.data_ptr() if checkpoint else None,
                                     act.exps.data_ptr() if checkpoint else None,
                                     _raw_stream(m.device)), "gq_gelu_forward")
    return h, act


def gq_gelu_backward(dh, act, approximate="none", need_output=False, stream=None):
    """du = dh gelu'(u) with u from its checkpoint; with need_output (du, gelu(u))."""
    d = _matrix(dh, "dh")
    rows, cols = d.shape
    form = _form(approximate)
    _covers(act, rows, cols, d.device)
    with _place(d.device, stream):
        du = torch.empty(dh.shape, dtype=dh.dtype, device=d.device)
        h = torch.empty(dh.shape, dtype=dh.dtype, device=d.device) if need_output else None
        _check(lib().gq_gelu_backward(d.data_ptr(), _IN_TYPES[d.dtype], rows, cols, _ld(d),
                                      act.codes.data_ptr(), act.exps.data_ptr(), form, du.data_ptr(),
                                      cols, h.data_ptr() if need_output else None, cols,
                                      _raw_stream(d.device)), "gq_gelu_backward")
    return (du, h) if need_output else du


def gq_linear_wgrad(dy, act, scale=None, shift=None, out_dtype=torch.float32, need_bias=True, ws=None,
                    stream=None):
    """(dw, dbias) of a linear layer from the gradient of its output (rows x outs) and the
    checkpoint of its input, or of that input's value before a per-column scale and shift (float32;
    a layer norm's weight and bias).  dw: outs x cols of out_dtype; dbias: float32, None without
    need_bias."""
    d = _matrix(dy, "dy")
    rows, outs = d.shape
    device = d.device
    _covers(act, rows, None, device)
    cols = act.cols
    if out_dtype not in _IN_TYPES:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if _vectors(cols, device, scale, shift) != F32:
        raise TypeError("scale and shift must be float32")
    with _place(device, stream):
        nbytes = lib().gq_linear_wgrad_workspace_bytes(d.data_ptr(), _IN_TYPES[d.dtype], rows, outs,
                                                       _ld(d), cols)
        ws = _workspace(ws, nbytes, device)
        dw = torch.empty((outs, cols), dtype=out_dtype, device=device)
        db = torch.empty(outs, dtype=torch.float32, device=device) if need_bias else None
        _check(lib().gq_linear_wgrad(
            d.data_ptr(), _IN_TYPES[d.dtype], rows, outs, _ld(d), act.codes.data_ptr(),
            act.exps.data_ptr(), cols, None if scale is None else scale.data_ptr(),
            None if shift is None else shift.data_ptr(), dw.data_ptr(), _IN_TYPES[out_dtype], cols,
            db.data_ptr() if need_bias else None, ws.data_ptr(), ws.numel() * ws.element_size(),
            _raw_stream(device)), "gq_linear_wgrad")
    return dw, db
