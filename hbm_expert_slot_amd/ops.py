"""Operators on 4-bit weights over torch tensors.

torch supplies device memory and streams; the work is done by the library's
HIP kernels.  Calls are asynchronous on `stream` (the current stream of the
tensors' device if None) and can be captured into a graph.
"""
import ctypes

import torch

from . import binding as B

_TYPE = {torch.float32: B.SC_DTYPE_F32, torch.bfloat16: B.SC_DTYPE_BF16, torch.float16: B.SC_DTYPE_F16}
_FORMAT = {"nvfp4": B.SC_FP4_NV, "mxfp4": B.SC_FP4_MX}
GROUP = {"nvfp4": 16, "mxfp4": 32}


class _On:
    """Makes `device`, and `stream` if one is given, current for the calls
    inside, and yields the raw stream: what a call allocates then belongs to
    the stream that it runs on."""

    __slots__ = ("device", "stream", "guard")

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError("the stream belongs to %s, the tensors to %s" % (stream.device, device))
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        if self.stream is not None:
            self.guard = torch.cuda.stream(self.stream)
        elif self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
        if self.guard is not None:
            self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _matrix(t, name, dtypes):
    _need(t.dim() == 2, "%s must have two dimensions" % name)
    _need(t.dtype in dtypes, "%s has type %s" % (name, t.dtype))
    _need(t.is_cuda, "%s must be on the GPU" % name)
    _need(t.shape[1] <= 1 or t.stride(1) == 1, "%s must be contiguous along its rows" % name)


def _ld(t):
    """Row stride; a single row counts as dense, whatever stride it has."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _check_ld(t, name):
    _need(t.shape[0] <= 1 or t.stride(0) >= t.shape[1], "%s has rows that overlap" % name)


class FP4Weight:
    """A matrix [rows, cols] in 4 bits.

    codes uint8 [rows, cols/2] (two E2M1 codes per byte, the even element low),
    scales uint8 [rows, cols/16] (E4M3, "nvfp4") or [rows, cols/32] (E8M0,
    "mxfp4"), global_scale fp32 with one element ("nvfp4"; None stands for 1).
    The tensors are referred to, not copied: they may be views into an expert
    blob."""

    def __init__(self, codes, scales, global_scale=None, fmt="nvfp4"):
        _need(fmt in _FORMAT, "unknown format %r" % (fmt,))
        for t, name in ((codes, "codes"), (scales, "scales")):
            _need(t.dim() == 2 and t.dtype == torch.uint8 and t.is_contiguous(),
                  "%s must be a contiguous two-dimensional uint8 tensor" % name)
            _need(t.is_cuda and t.device == codes.device, "%s must be on the GPU, with the codes" % name)
        rows, cols = codes.shape[0], 2 * codes.shape[1]
        _need(cols > 0 and cols % GROUP[fmt] == 0, "columns must be a positive multiple of %d" % GROUP[fmt])
        _need(tuple(scales.shape) == (rows, cols // GROUP[fmt]), "scales have shape %s" % (tuple(scales.shape),))
        if global_scale is not None:
            _need(fmt == "nvfp4", "only nvfp4 has a global scale")
            _need(global_scale.dtype == torch.float32 and global_scale.numel() == 1
                  and global_scale.device == codes.device, "global_scale must be one float32 with the codes")
        self.codes, self.scales, self.global_scale, self.fmt = codes, scales, global_scale, fmt
        self.rows, self.cols, self.device = rows, cols, codes.device
        self._c = B.sc_fp4_matrix(_FORMAT[fmt], rows, cols, codes.data_ptr(), scales.data_ptr(),
                                  None if global_scale is None else global_scale.data_ptr())
        self._ref = ctypes.byref(self._c)

    @property
    def shape(self):
        return (self.rows, self.cols)

    @staticmethod
    def empty(rows, cols, fmt="nvfp4", device="cuda"):
        _need(fmt in _FORMAT, "unknown format %r" % (fmt,))
        _need(rows >= 0 and cols > 0 and cols % GROUP[fmt] == 0,
              "columns must be a positive multiple of %d" % GROUP[fmt])
        u8 = dict(dtype=torch.uint8, device=device)
        gs = torch.ones(1, dtype=torch.float32, device=device) if fmt == "nvfp4" else None
        return FP4Weight(torch.empty((rows, cols // 2), **u8), torch.empty((rows, cols // GROUP[fmt]), **u8), gs, fmt)


def fp4_quantize(w, fmt="nvfp4", global_scale=None, out=None, stream=None):
    """Quantise w [rows, cols] (float32, bfloat16 or float16) to 4 bits.

    "nvfp4": with global_scale (one positive fp32 on the device) that scale is
    used, without it max|w| / 2688.  Codes and scales are the nearest to the
    exact quotients, ties to even; a group with an infinity or NaN reads back as
    NaN.  `out` is a FP4Weight to write (its global_scale too)."""
    _matrix(w, "w", _TYPE)
    _check_ld(w, "w")
    _need(fmt in _FORMAT, "unknown format %r" % (fmt,))
    rows, cols = w.shape
    _need(cols > 0 and cols % GROUP[fmt] == 0, "columns must be a positive multiple of %d" % GROUP[fmt])
    _need(global_scale is None or fmt == "nvfp4", "only nvfp4 has a global scale")
    dev = w.device
    if global_scale is not None:
        _need(global_scale.dtype == torch.float32 and global_scale.numel() == 1 and global_scale.device == dev,
              "global_scale must be one float32 on the device of w")
    with _On(dev, stream) as s:
        if out is None:
            u8 = dict(dtype=torch.uint8, device=dev)
            gs = global_scale
            if fmt == "nvfp4" and gs is None:
                gs = torch.ones(1, dtype=torch.float32, device=dev) if rows == 0 else \
                    torch.empty(1, dtype=torch.float32, device=dev)
            out = FP4Weight(torch.empty((rows, cols // 2), **u8), torch.empty((rows, cols // GROUP[fmt]), **u8),
                            gs, fmt)
        else:
            _need(out.shape == (rows, cols) and out.fmt == fmt and out.device == dev, "out does not fit w")
            _need(fmt != "nvfp4" or out.global_scale is not None, "out needs a global_scale")
            if global_scale is not None and global_scale.data_ptr() != out.global_scale.data_ptr():
                raise ValueError("out.global_scale must be the given global_scale")
        ws = None
        if fmt == "nvfp4" and global_scale is None:
            ws = torch.empty(B.SC_FP4_QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
        B.fp4_quantize(w.data_ptr(), _TYPE[w.dtype], _ld(w), out._ref, 0 if global_scale is None else 1,
                       None if ws is None else ws.data_ptr(), s)
    return out


def fp4_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values q stands for, [rows, cols] of `dtype`."""
    dev = q.device
    with _On(dev, stream) as s:
        if out is None:
            _need(dtype in _TYPE, "unsupported type %s" % (dtype,))
            out = torch.empty((q.rows, q.cols), dtype=dtype, device=dev)
        else:
            _matrix(out, "out", _TYPE)
            _check_ld(out, "out")
            _need(tuple(out.shape) == q.shape and out.device == dev, "out does not fit")
        B.fp4_dequantize(q._ref, out.data_ptr(), _TYPE[out.dtype], _ld(out), s)
    return out


def fp4_linear(x, q, bias=None, out_dtype=None, out=None, stream=None):
    """x [M, cols] (bfloat16 or float16) times the transpose of q [rows, cols],
    plus bias fp32 [rows]; [M, rows] of out_dtype (default: x's type)."""
    _matrix(x, "x", (torch.bfloat16, torch.float16))
    dev = x.device
    M = x.shape[0]
    _need(x.shape[1] == q.cols and q.device == dev, "x [%d, %d] does not fit a weight of %d columns on %s"
          % (M, x.shape[1], q.cols, q.device))
    _check_ld(x, "x")
    if bias is not None:
        _need(bias.dtype == torch.float32 and tuple(bias.shape) == (q.rows,) and bias.is_contiguous()
              and bias.device == dev, "bias must be a contiguous float32 vector of %d on %s" % (q.rows, dev))
    with _On(dev, stream) as s:
        if out is None:
            dt = x.dtype if out_dtype is None else out_dtype
            _need(dt in _TYPE, "unsupported type %s" % (dt,))
            out = torch.empty((M, q.rows), dtype=dt, device=dev)
        else:
            _matrix(out, "out", _TYPE)
            _check_ld(out, "out")
            _need(tuple(out.shape) == (M, q.rows) and out.device == dev, "out does not fit")
            _need(out_dtype is None or out.dtype == out_dtype, "out has type %s" % (out.dtype,))
        B.fp4_linear(q._ref, x.data_ptr(), _TYPE[x.dtype], _ld(x), M, None if bias is None else bias.data_ptr(),
                     out.data_ptr(), _TYPE[out.dtype], _ld(out), s)
    return out
