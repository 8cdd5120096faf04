"""Operators on 4-bit weights over torch tensors.

torch supplies device memory and streams; the work is done by the library's
HIP kernels.  The operators are for inference: their results have no gradient,
and going backward through one raises NotImplementedError.
Calls are asynchronous on `stream` (the current stream of the
tensors' device if None) and can be captured into a graph.  What a call
allocates belongs to its stream.  Tensors given to a call with `stream` may be
dropped as soon as it returns: their memory is not used again before the
stream is done with it.  A captured graph does not keep its tensors: that is
the caller's part.
"""
import ctypes

import torch

from . import binding as B

_TYPE = {torch.float32: B.SC_DTYPE_F32, torch.bfloat16: B.SC_DTYPE_BF16, torch.float16: B.SC_DTYPE_F16}
_FORMAT = {"nvfp4": B.SC_FP4_NV, "mxfp4": B.SC_FP4_MX}
GROUP = {"nvfp4": 16, "mxfp4": 32}


def _stream_handle(index):
    return torch.cuda.current_stream(index).cuda_stream


# the handle alone, where torch has it: torch.cuda.current_stream also makes an object, which costs 1.8 us
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)


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
        return _raw_stream(self.device.index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _record(stream, *tensors):
    """The memory of the tensors is not given out again before what `stream` has been given is done."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


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


class _ForInference(torch.autograd.Function):
    """call(), on behalf of inputs some of which require a gradient."""

    @staticmethod
    def forward(ctx, name, call, *inputs):
        ctx.name = name
        return call()

    @staticmethod
    def backward(ctx, *grads):
        raise NotImplementedError("%s is for inference: it has no gradient" % ctx.name)


def _wants_grad(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


class _Fixed:
    """Objects that hand addresses to the library: what those belong to cannot be
    assigned again (assigning would leave the library with the old ones)."""

    _fixed = frozenset()

    def __setattr__(self, name, value):
        if name in self._fixed and name in self.__dict__:
            raise AttributeError("%s of a %s is fixed when it is made" % (name, type(self).__name__))
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._fixed:
            raise AttributeError("%s of a %s is fixed when it is made" % (name, type(self).__name__))
        object.__delattr__(self, name)


class FP4Weight(_Fixed):
    """A matrix [rows, cols] in 4 bits.

    codes uint8 [rows, cols/2] (two E2M1 codes per byte, the even element low),
    scales uint8 [rows, cols/16] (E4M3, "nvfp4") or [rows, cols/32] (E8M0,
    "mxfp4"), global_scale fp32 with one element ("nvfp4"; None stands for 1).
    The tensors are referred to, not copied: they may be views into an expert
    blob.  They can be written to, but not exchanged: the weight keeps the memory
    it was made of, also where a tensor is given other storage later."""

    _fixed = frozenset(("codes", "scales", "global_scale", "fmt", "rows", "cols", "device", "_memory", "_c", "_ref"))

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
        memory = [codes.untyped_storage(), scales.untyped_storage()]
        if global_scale is not None:
            memory.append(global_scale.untyped_storage())
        c = B.sc_fp4_matrix(_FORMAT[fmt], rows, cols, codes.data_ptr(), scales.data_ptr(),
                            None if global_scale is None else global_scale.data_ptr())
        # all at once, past the check of each name
        self.__dict__.update(codes=codes, scales=scales, global_scale=global_scale, fmt=fmt, rows=rows, cols=cols,
                             device=codes.device, _memory=memory, _c=c, _ref=ctypes.byref(c))

    @property
    def shape(self):
        return (self.rows, self.cols)

    def _record(self, stream):
        for m in self._memory:
            _record(stream, torch.empty(0, dtype=torch.uint8, device=self.device).set_(m))

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
    if stream is not None:
        _record(stream, w)
        out._record(stream)
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
    if stream is not None:
        _record(stream, out)
        q._record(stream)
    return out


def fp4_linear(x, q, bias=None, out_dtype=None, out=None, stream=None):
    """x [M, cols] (bfloat16 or float16) times the transpose of q [rows, cols],
    plus bias fp32 [rows]; [M, rows] of out_dtype (default: x's type), or in out,
    which must not overlap x (and takes no part in a gradient)."""
    if (x.requires_grad or bias is not None) and out is None and _wants_grad(x, bias):
        return _ForInference.apply("fp4_linear", lambda: fp4_linear(x, q, bias, out_dtype, None, stream), x, bias)
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
    if stream is not None:
        _record(stream, x, bias, out)
        q._record(stream)
    return out


def blob_bytes(hidden, inter):
    """Bytes of one expert's blob."""
    return 27 * hidden * inter // 16


def expert_matrices(blob, hidden, inter, global_scales):
    """The two matrices of an expert blob (uint8 [blob_bytes]) as FP4Weight views: w13
    [2 inter, hidden] (gate rows, then up rows) and w2 [hidden, inter], with
    the entries of global_scales fp32 [2]."""
    _need(blob.dim() == 1 and blob.dtype == torch.uint8 and blob.numel() == blob_bytes(hidden, inter)
          and hidden % 64 == 0 and inter % 64 == 0, "blob does not hold an expert of %d x %d" % (hidden, inter))
    a, b, c = inter * hidden, inter * hidden // 8, hidden * inter // 2
    w13 = FP4Weight(blob[:a].view(2 * inter, hidden // 2), blob[a:a + b].view(2 * inter, hidden // 16),
                    global_scales[0:1])
    w2 = FP4Weight(blob[a + b:a + b + c].view(hidden, inter // 2), blob[a + b + c:].view(hidden, inter // 16),
                   global_scales[1:2])
    return w13, w2


class MoELayer(_Fixed):
    """A whole mixture-of-experts layer for up to `max_rows` (16) tokens a call.

    router bf16 [E, hidden]; blobs uint8 [E, blob_bytes] and global_scales fp32
    [E, 2] hold the routed experts (the layout of the slot cache, all resident
    in HBM); shared_blob and shared_global_scales [2] the shared expert, if any
    (its inner size follows from the blob's).  score "softmax" or "sigmoid" (with
    score_bias fp32 [E] added for the choice only); routed_scale multiplies the
    routed sum.  The tensors are referred to, not copied; they can be written to,
    but the layer keeps the memory it was made of.

    The layer owns a workspace: calls have to be ordered with each other (one
    stream, or streams the caller orders); use one layer object per stream
    otherwise.  A call that waits for over a second because another one runs on
    the workspace gives up and returns NaN; prepare() makes the workspace ready
    again once both are done.  A layer may be dropped while calls are under way, but not while a
    captured graph is to be replayed."""

    _fixed = frozenset(("hidden", "inter", "n_experts", "top_k", "shared_inter", "max_rows", "device", "workspace",
                        "_memory", "_streams", "_ws", "_cfg", "_cref", "_w", "_wref"))

    def __init__(self, hidden, inter, top_k, router, blobs, global_scales, shared_blob=None,
                 shared_global_scales=None, score="softmax", score_bias=None, routed_scale=1.0, max_rows=16):
        _need(score in ("softmax", "sigmoid"), "unknown score %r" % (score,))
        _need(router.dim() == 2 and router.shape[1] == hidden, "router must be [experts, hidden]")
        _need(hidden > 0 and inter > 0, "hidden and inter must be positive")
        E, dev = router.shape[0], router.device

        def dense(t, name, dtype, shape):
            _need(t.dtype == dtype and tuple(t.shape) == shape and t.is_contiguous(),
                  "%s must be a contiguous %s tensor of shape %s" % (name, dtype, shape))
            _need(t.is_cuda and t.device == dev, "%s must be on the GPU, with the router" % name)

        dense(router, "router", torch.bfloat16, (E, hidden))
        dense(blobs, "blobs", torch.uint8, (E, blob_bytes(hidden, inter)))
        dense(global_scales, "global_scales", torch.float32, (E, 2))
        shared_inter = 0
        if shared_blob is not None:
            _need(shared_global_scales is not None, "the shared expert needs shared_global_scales")
            shared_inter = shared_blob.numel() * 16 // (27 * hidden)
            dense(shared_blob, "shared_blob", torch.uint8, (blob_bytes(hidden, shared_inter),))
            dense(shared_global_scales, "shared_global_scales", torch.float32, (2,))
            _need(shared_inter > 0, "shared_blob is empty")
        if score_bias is not None:
            _need(score == "sigmoid", "only the sigmoid score has a bias")
            dense(score_bias, "score_bias", torch.float32, (E,))
        self._cfg = B.sc_moe_config(hidden, inter, E, top_k, shared_inter, max_rows,
                                    B.SC_SCORE_SIGMOID if score == "sigmoid" else B.SC_SCORE_SOFTMAX, routed_scale)
        self._cref = ctypes.byref(self._cfg)
        n = B.moe_layer_workspace_bytes(self._cref)

        def ptr(t):
            return None if t is None else t.data_ptr()

        self._memory = [t.detach() for t in (router, blobs, global_scales, shared_blob, shared_global_scales, score_bias)
                        if t is not None]
        self._grads = [t for t in (router, global_scales, shared_global_scales, score_bias) if t is not None]
        self._streams = set()        # that the memory is recorded on
        self._w = B.sc_moe_weights(ptr(router), ptr(score_bias), ptr(blobs), ptr(global_scales), ptr(shared_blob),
                                   ptr(shared_global_scales))
        self._wref = ctypes.byref(self._w)
        self.hidden, self.inter, self.n_experts, self.top_k = hidden, inter, E, top_k
        self.shared_inter, self.max_rows, self.device = shared_inter, max_rows, dev
        with _On(dev, None) as s:
            self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)
            self._memory.append(self.workspace.detach())
            self._ws = self.workspace.data_ptr()
            B.moe_layer_prepare(self._cref, self._ws, s)
            torch.cuda.current_stream(dev).synchronize()

    def _used_on(self, s):
        """The layer may be dropped while the current stream (raw: s, not in _streams yet) works on it."""
        _record(torch.cuda.current_stream(self.device), *self._memory)
        self._streams.add(s)

    def prepare(self, stream=None):
        """Clears the workspace's control words, as the constructor does: needed only after calls that ran on
        the layer at once, when all of them are done."""
        with _On(self.device, stream) as s:
            B.moe_layer_prepare(self._cref, self._ws, s)
            if s not in self._streams:
                self._used_on(s)

    def forward(self, x, out_dtype=torch.float32, out=None, ids=None, weights=None, stream=None):
        """y [M, hidden] for x bf16 [M, hidden], M <= max_rows.  out_dtype float32 or bfloat16.  ids int32 and
        weights float32 [M, top_k], if given, receive the picks and their weights in rank order.  out, if given,
        must not overlap x (and takes no part in a gradient)."""
        if out is None and _wants_grad(x, *self._grads):
            return _ForInference.apply("MoELayer.forward",
                                       lambda: self.forward(x, out_dtype, None, ids, weights, stream), x, *self._grads)
        _matrix(x, "x", (torch.bfloat16,))
        _check_ld(x, "x")
        M, dev = x.shape[0], self.device
        _need(x.shape[1] == self.hidden and x.device == dev, "x does not fit the layer")
        _need(M <= self.max_rows, "at most %d rows" % self.max_rows)
        for t, name, dt in ((ids, "ids", torch.int32), (weights, "weights", torch.float32)):
            _need(t is None or (t.dtype == dt and tuple(t.shape) == (M, self.top_k) and t.is_contiguous()
                                and t.device == dev), "%s must be a contiguous [M, top_k] %s tensor" % (name, dt))
        with _On(dev, stream) as s:
            if out is None:
                _need(out_dtype in (torch.float32, torch.bfloat16), "unsupported type %s" % (out_dtype,))
                out = torch.empty((M, self.hidden), dtype=out_dtype, device=dev)
            else:
                _matrix(out, "out", (torch.float32, torch.bfloat16))
                _check_ld(out, "out")
                _need(tuple(out.shape) == (M, self.hidden) and out.device == dev, "out does not fit")
            B.moe_layer_forward(self._cref, self._wref, self._ws, x.data_ptr(), _ld(x), M,
                                out.data_ptr(), _TYPE[out.dtype], _ld(out), None if ids is None else ids.data_ptr(),
                                None if weights is None else weights.data_ptr(), s)
            if s not in self._streams:
                self._used_on(s)
        if stream is not None:
            _record(stream, x, out, ids, weights)
        return out
