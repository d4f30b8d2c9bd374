"""Torch-facing row operators: residual addition + norm, linear, E4M3 rows.

Rows are the last dimension's vectors: a tensor [..., cols] is taken as rows of
cols elements. A round's activations [S+1][C][heads][d] are viewed as
[(S+1) * C][heads * d]; the live slots are its first rows, so ``x[:n]`` of such a
view (or one slot's rows) is what a fill round passes. Every computation runs in
libwf's kernels; PyTorch allocates outputs that the caller does not give.

The calls enqueue on ``stream`` (default: the tensors' device's current stream)
and do not synchronise. They compute no gradients and refuse tensors that want
them while gradients are recorded, and tensors that carry a forward-mode tangent.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib
import importlib.util
import math
import struct
import warnings
from typing import Optional, Tuple, Union

import torch
from torch.autograd.forward_ad import unpack_dual

from . import wf as _wf
from .wf import WfError

_TYPES = {torch.bfloat16: _wf.WF_DTYPE_BF16, torch.float32: _wf.WF_DTYPE_F32}
_ACTS = {"none": _wf.WF_ACT_NONE, "gelu": _wf.WF_ACT_GELU, "silu": _wf.WF_ACT_SILU}


# The current device, and its current stream's handle, without the objects around them.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class E4M3Rows:
    """Rows held as E4M3 codes with a power-of-two scale per 32 columns.

    codes  : float8_e4m3fn [rows, cols], cols a multiple of 32, unit column stride
    scales : uint8, wf_scale_bytes(rows, cols) bytes: e + 127 of each block (a
             block's values are code * 2^e), in tiles of 128 rows x 4 blocks
             (include/wf.h gives the order)
    """

    __slots__ = ("codes", "scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 2 or codes.dtype != torch.float8_e4m3fn:
            raise ValueError("codes must be a float8_e4m3fn tensor [rows, cols]")
        if scales.dtype != torch.uint8 or not scales.is_contiguous():
            raise ValueError("scales must be a contiguous uint8 tensor")
        rows, cols = codes.shape
        if cols % 32 or cols == 0:
            raise ValueError("E4M3 rows need a multiple of 32 columns")
        if scales.numel() < (rows + 127) // 128 * ((cols + 127) // 128) * 512:
            raise ValueError("scales has fewer than wf_scale_bytes(rows, cols) bytes")
        if scales.device != codes.device:
            raise ValueError("codes and scales must be on one device")
        self.codes, self.scales = codes, scales

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "E4M3Rows":
        n = _wf.wf_scale_bytes(rows, cols)
        return cls(torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device),
                   torch.empty(n, dtype=torch.uint8, device=device))

    @property
    def shape(self) -> torch.Size:
        return self.codes.shape

    @property
    def device(self) -> torch.device:
        return self.codes.device

    requires_grad = False

    def get_device(self) -> int:
        return self.codes.get_device()

    def first(self, rows: int) -> "E4M3Rows":
        """The first rows, sharing memory."""
        if not 0 <= rows <= self.codes.shape[0]:
            raise ValueError(f"there are {self.codes.shape[0]} rows, not {rows}")
        return E4M3Rows(self.codes[:rows], self.scales)

    def span(self, start: int, stop: int) -> "E4M3Rows":
        """Rows [start, stop), sharing memory; start is a multiple of 128 (the scales' tiles)."""
        rows, cols = self.codes.shape
        if start % 128 or not 0 <= start <= stop <= rows:
            raise ValueError("a span of E4M3 rows starts at a multiple of 128 inside them")
        return E4M3Rows(self.codes[start:stop], self.scales[start // 128 * ((cols + 127) // 128) * 512:])

    def dequantize(self, out: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                   stream=None) -> torch.Tensor:
        """The values these rows stand for, as bf16 or fp32 (exact in both)."""
        if _fast is not None and out is None and stream is None and dtype in _TYPES:
            r = _fast.dequantize_rows(self.codes, self.scales, dtype is torch.float32)
            if r is not NotImplemented:
                return r if type(r) is not int else _check(r, "wf_dequantize_rows")
        raw = _here(stream, self, out)
        if raw is None:
            with _elsewhere(self.device, stream):
                return self.dequantize(out, dtype)
        if out is None:
            out = self.codes.new_empty(self.codes.shape, dtype=dtype)
        _check(_dequantize(_rows(self), _rows(out), raw), "wf_dequantize_rows")
        return out


Operand = Union[torch.Tensor, E4M3Rows]


# One wf_rows struct (native alignment, padded to its size).
_pack = struct.Struct("PPqqqi0q").pack
_E4M3 = _wf.WF_DTYPE_FP8_E4M3


def _rows(t: Optional[Operand]) -> Optional[bytes]:
    """The wf_rows struct of an operand, as bytes; a view, never a copy."""
    if t is None:
        return None
    if type(t) is E4M3Rows:
        c = t.codes
        rows, cols = c.shape
        ld, unit = c.stride()
        if unit != 1 or (rows > 1 and ld < cols):
            raise ValueError("rows must have unit column stride and not share memory")
        return _pack(c.data_ptr(), t.scales.data_ptr(), rows, cols, ld if ld > cols else cols, _E4M3)
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"rows must be bfloat16, float32 or E4M3Rows, not {t.dtype}")
    shape = t.shape
    cols = shape[-1] if shape else 0
    if cols == 0:
        raise ValueError("rows must have at least one column")
    if t.is_contiguous():
        return _pack(t.data_ptr(), 0, t.numel() // cols, cols, cols, code)
    if len(shape) == 2 and (t.stride(1) == 1 or cols == 1):
        rows, ld = shape[0], t.stride(0)
        if rows > 1 and ld < cols:
            raise ValueError("rows that share memory (an expanded tensor) are not supported")
        return _pack(t.data_ptr(), 0, rows, cols, max(ld, cols), code)
    raise ValueError("rows must be contiguous, or 2-D with unit column stride")


def _entry(name: str):
    """The library's entry point, taking wf_rows structs as bytes: building a ctypes
    Structure for each operand costs more than the launch."""
    fn = _wf.lib()[name]
    P = ctypes.c_void_p
    kinds = {"r": ctypes.c_char_p, "p": P, "i": ctypes.c_int32, "f": ctypes.c_float}
    fn.argtypes = [kinds[k] for k in {"wf_quantize_rows": "rrp", "wf_dequantize_rows": "rrp",
                                      "wf_add_rms_norm": "rrpfrrp", "wf_linear": "rrpirrp"}[name]]
    fn.restype = ctypes.c_int32
    return fn


_quantize, _dequantize = _entry("wf_quantize_rows"), _entry("wf_dequantize_rows")
_norm, _linear = _entry("wf_add_rms_norm"), _entry("wf_linear")

def _load_fast():
    """The compiled common case of the calls below, or None.

    It is the same library calls with less of the host's time, for contiguous tensors on the current
    device, outputs to be allocated and the current stream; it answers NotImplemented where the code
    below has to check, refuse or convert. Without it that code serves every call, so a module that
    was built for another torch, or does not load, is left alone."""
    name = __package__ + "._rows_bind"
    if importlib.util.find_spec(name) is None:
        return None
    try:
        fast = importlib.import_module(name)
        built = fast.torch_version
    except (ImportError, OSError, SystemError, AttributeError) as e:
        why = str(e)
    else:
        if built == str(torch.__version__):
            fast.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (_linear, _norm, _quantize, _dequantize)))
            return fast
        why = f"it was built for torch {built}, this is {torch.__version__}"
    warnings.warn(f"{name} is not used ({why}): small row operators take more host time until "
                  "chunk_causal_wavefront_b200/build.py has run", RuntimeWarning, stacklevel=2)
    return None


_fast = _load_fast()


def _made(codes: torch.Tensor, scales: torch.Tensor) -> "E4M3Rows":
    out = E4M3Rows.__new__(E4M3Rows)
    out.codes, out.scales = codes, scales
    return out


def _check(status: int, what: str) -> None:
    if status != _wf.WF_OK:
        raise WfError(status, what)


def refuse_gradients(what: str, *operands: Optional[Operand]) -> None:
    """Raises if an operand wants a gradient that nothing here would compute: one that records, or a
    dual tensor, whose tangent the result would lose (also under torch.no_grad())."""
    recording = torch.is_grad_enabled()
    for t in operands:
        if t is None:
            continue
        if isinstance(t, E4M3Rows):
            t = t.codes
        if recording and t.requires_grad:
            raise ValueError(f"{what} compute no gradients: call them under torch.no_grad()")
        if unpack_dual(t).tangent is not None:
            raise ValueError(f"{what} compute no tangents: give them the primal of a dual tensor")


def _here(stream, x, *others) -> Optional[int]:
    """Checks that everything is on one CUDA device. The raw current stream if that device is
    current and no stream is given; else None: the call goes through _elsewhere."""
    index = x.get_device()
    if index < 0:
        raise ValueError("row operators need CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on one device: got {x.device} and {t.device}")
    refuse_gradients("row operators", x, *others)
    if stream is not None:
        if stream.device != x.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
        return None
    return _raw_stream(index) if index == _current_device() else None


@contextlib.contextmanager
def _elsewhere(device, stream):
    """Makes the tensors' device current, and the given stream, so that outputs allocated
    inside belong to it."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _vector(v: torch.Tensor, n: int, name: str) -> int:
    if v.dtype != torch.float32 or v.shape != (n,) or not v.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 vector of {n} elements")
    return v.data_ptr()


def _given(out: Operand, shape, out_dtype) -> Operand:
    """The caller's output after a check of its shape (E4M3 rows: leading dimensions flattened)."""
    if out_dtype is not None:
        raise ValueError("give out or out_dtype, not both")
    want = (math.prod(shape[:-1]), shape[-1]) if isinstance(out, E4M3Rows) else tuple(shape)
    if tuple(out.shape) != want:
        raise ValueError(f"out has shape {tuple(out.shape)}, not {want}")
    return out


def _new(like: torch.Tensor, shape, out_dtype, default: torch.dtype) -> Operand:
    """A new output on the device of `like`."""
    if out_dtype is None or out_dtype is default:
        return like.new_empty(shape) if like.dtype is default else like.new_empty(shape, dtype=default)
    if out_dtype == "e4m3":
        rows, cols = math.prod(shape[:-1]), shape[-1]
        if cols % 32:
            raise ValueError("E4M3 rows need a multiple of 32 columns")
        return _made(like.new_empty((rows, cols), dtype=torch.float8_e4m3fn),
                     like.new_empty((rows + 127) // 128 * ((cols + 127) // 128) * 512, dtype=torch.uint8))
    raise ValueError(f"out_dtype must be {default} (the default) or 'e4m3'")


def _packed_like(x: torch.Tensor) -> torch.Tensor:
    return x.new_empty(x.shape)


def quantize_rows(x: torch.Tensor, out: Optional[E4M3Rows] = None, stream=None) -> E4M3Rows:
    """x [..., cols] in bf16 or fp32 as E4M3 rows (leading dimensions flattened)."""
    if _fast is not None and out is None and stream is None:
        r = _fast.quantize_rows(x)
        if r is not NotImplemented:
            return _made(*r) if type(r) is not int else _check(r, "wf_quantize_rows")
    raw = _here(stream, x, out)
    if raw is None:
        with _elsewhere(x.device, stream):
            return quantize_rows(x, out)
    out = _new(x, x.shape, "e4m3", x.dtype) if out is None else _given(out, x.shape, None)
    _check(_quantize(_rows(x), _rows(out), raw), "wf_quantize_rows")
    return out


def add_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                 residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 out: Optional[Operand] = None, sum_out: Optional[torch.Tensor] = None,
                 out_dtype=None, stream=None) -> Union[Operand, Tuple[Operand, torch.Tensor]]:
    """s = x + residual; out = s / sqrt(mean(s^2) + eps) * weight, row by row.

    Computed in fp32 (the sum of squares in 64 bits): a row with a value beyond 2^63
    or so has an infinite mean, and out is 0 there.

    Without a residual returns out, with one (out, s). out has x's type, or is
    E4M3Rows with out_dtype="e4m3" (or out=E4M3Rows). sum_out may be x or
    residual: the residual stream is then updated in place. weight is float32.
    """
    if (_fast is not None and out is None and sum_out is None and stream is None
            and (out_dtype is None or out_dtype == "e4m3")):
        r = _fast.add_rms_norm(x, weight, residual, eps, out_dtype is not None)
        if r is not NotImplemented:
            if type(r) is int:
                _check(r, "wf_add_rms_norm")
            if out_dtype is None:
                return r
            return _made(*r) if residual is None else (_made(r[0], r[1]), r[2])
    shape = x.shape
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
    elif residual.shape != shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(shape)}")
    if sum_out is not None and sum_out.shape != shape:
        raise ValueError(f"sum_out has shape {tuple(sum_out.shape)}, x {tuple(shape)}")
    raw = _here(stream, x, weight, residual, out, sum_out)
    if raw is None:
        with _elsewhere(x.device, stream):
            return add_rms_norm(x, weight, residual=residual, eps=eps, out=out, sum_out=sum_out,
                                out_dtype=out_dtype)
    xr = _rows(x)
    w = None if weight is None else _vector(weight, shape[-1], "weight")
    if x.is_contiguous():                     # new rows have x's layout
        new = torch.empty_like
    else:
        new = _packed_like
    if out is not None:
        _given(out, shape, out_dtype)
    elif out_dtype is None or out_dtype is x.dtype:
        out = new(x)
    else:
        out = _new(x, shape, out_dtype, x.dtype)
    if residual is None:
        _check(_norm(xr, None, w, eps, None, _rows(out), raw), "wf_add_rms_norm")
        return out
    if sum_out is None:
        sum_out = new(x)
    _check(_norm(xr, _rows(residual), w, eps, _rows(sum_out), _rows(out), raw), "wf_add_rms_norm")
    return out, sum_out


def linear(x: Operand, w: Operand, bias: Optional[torch.Tensor] = None, *, act: str = "none",
           residual: Optional[torch.Tensor] = None, out: Optional[Operand] = None,
           out_dtype=None, stream=None) -> Operand:
    """act(x w^T + bias) + residual on the tensor cores, accumulated in fp32.

    x [..., K] and w [N, K] are both bf16 or both E4M3Rows, their rows at multiples of
    16 bytes (contiguous bf16: K a multiple of 8); bias is float32 [N]; act is "none",
    "gelu" (tanh form) or "silu". The result is bf16 [..., N], or E4M3Rows with
    out_dtype="e4m3" (or out=E4M3Rows), then without a residual. out may be residual
    itself.
    """
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    if (_fast is not None and out is None and stream is None
            and (out_dtype is None or out_dtype == "e4m3")):
        if type(x) is E4M3Rows and type(w) is E4M3Rows:
            r = _fast.linear(x.codes, x.scales, w.codes, w.scales, bias, code, residual, out_dtype is not None)
        else:
            r = _fast.linear(x, None, w, None, bias, code, residual, out_dtype is not None)
        if r is not NotImplemented:
            if type(r) is int:
                _check(r, "wf_linear")
            return r if out_dtype is None else _made(*r)
    xs, ws = x.shape, w.shape
    if len(ws) != 2 or not xs or xs[-1] != ws[1]:
        raise ValueError(f"shapes {tuple(xs)} and {tuple(ws)} do not give x w^T")
    shape = (*xs[:-1], ws[0])
    if residual is not None and residual.shape != shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, not {shape}")
    raw = _here(stream, x, w, bias, residual, out)
    if raw is None:
        with _elsewhere(x.device, stream):
            return linear(x, w, bias, act=act, residual=residual, out=out, out_dtype=out_dtype)
    b = None if bias is None else _vector(bias, ws[0], "bias")
    if out is None:
        out = _new(x.codes if type(x) is E4M3Rows else x, shape, out_dtype, torch.bfloat16)
    else:
        _given(out, shape, out_dtype)
    _check(_linear(_rows(x), _rows(w), b, code, _rows(residual), _rows(out), raw), "wf_linear")
    return out


def rows_check_status(device=None, stream=None) -> int:
    """Synchronise, then return and clear the device's row-operator status."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        s = torch.cuda.current_stream(device) if stream is None else stream
        return _wf.wf_rows_check_status(s.cuda_stream)
