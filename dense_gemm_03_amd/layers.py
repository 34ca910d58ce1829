"""Linear layers over torch tensors: ``linear`` and ``grouped_linear`` (products
with bias, activation and residual, dense or grouped by expert) and their
gradients ``linear_grad`` and ``grouped_linear_grad``; a thin binding over
``include/gemm_linear.h``.  Like the rest of the package they take no part in
torch's autograd: outputs carry no graph, whatever ``requires_grad`` says, and the
backward pass is the ``*_grad`` functions.  The C entry points are here under their own names
(``gemm_linear*``), taking parameters, device pointers and a stream."""
from __future__ import annotations

import ctypes

GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_GELU_TANH, GEMM_ACT_SILU = range(5)
ACTIVATIONS = {"none": GEMM_ACT_NONE, "relu": GEMM_ACT_RELU, "gelu": GEMM_ACT_GELU,
               "gelu_tanh": GEMM_ACT_GELU_TANH, "silu": GEMM_ACT_SILU}


class LinearParams(ctypes.Structure):
    """gemm_linear_params of include/gemm_linear.h."""
    _fields_ = [("dtype", ctypes.c_int32), ("dtype_y", ctypes.c_int32),
                ("dtype_bias", ctypes.c_int32), ("transw", ctypes.c_int32),
                ("act", ctypes.c_int32), ("alpha", ctypes.c_float)] + \
        [(name, ctypes.c_int64) for name in (
            "rows", "N", "K", "groups", "ldx", "ldw", "ldy", "ldr", "ldp", "stride_w",
            "stride_bias")]


class LinearGradOutputs(ctypes.Structure):
    """gemm_linear_grad_outputs of include/gemm_linear.h."""
    _fields_ = [("dtype_dx", ctypes.c_int32), ("dtype_dw", ctypes.c_int32), ("beta", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("lddx", ctypes.c_int64), ("lddw", ctypes.c_int64),
                ("stride_dw", ctypes.c_int64)]


_i64, _p, _int, _f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_pl = ctypes.POINTER(LinearParams)
_pg = ctypes.POINTER(LinearGradOutputs)
# Every symbol include/gemm_linear.h declares, with its ctypes signature.
SIGNATURES = {
    "gemm_linear_workspace_size": (_i64, [_pl]),
    "gemm_linear": (_int, [_pl, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p]),
    "gemm_linear_act_grad_workspace_size": (_i64, [_pl]),
    "gemm_linear_act_grad": (_int, [_pl, _p, _i64, _p, _p, _p, _i64, _p, _p, _i64, _p]),
    "gemm_linear_weight_grad_workspace_size": (_i64, [_pl]),
    "gemm_linear_weight_grad": (_int, [_pl, _p, _p, _p, _int, _f, _p, _p, _i64, _p]),
    "gemm_linear_grad_workspace_size": (_i64, [_pl, _pg, _int, _int, _int]),
    "gemm_linear_grad": (_int, [_pl, _pg] + [_p] * 9 + [_i64, _p]),
    "gemm_linear_num_configs": (_int, [_int]),
    "gemm_linear_config_name": (ctypes.c_char_p, [_int, _int]),
    "gemm_linear_config_forms": (_int, [_int, _int]),
    "gemm_linear_select_config": (_int, [_pl, _int]),
    "gemm_linear_force_config": (_int, [_int, _int]),
}


_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load_library
        _lib = load_library()
    return _lib


def _status(rc):
    if rc != 0:
        from . import GemmError
        raise GemmError(rc)


# ---------------------------------------------------------------- C names --

def gemm_linear_workspace_size(params) -> int:
    return _library().gemm_linear_workspace_size(params)


def gemm_linear(params, x, w, offsets, bias, residual, pre, y, workspace, workspace_bytes,
                stream=None) -> int:
    return _library().gemm_linear(params, x, w, offsets, bias, residual, pre, y, workspace,
                                  workspace_bytes, stream)


def gemm_linear_act_grad_workspace_size(params) -> int:
    return _library().gemm_linear_act_grad_workspace_size(params)


def gemm_linear_act_grad(params, dy, lddy, pre, offsets, dz, lddz, dbias, workspace,
                         workspace_bytes, stream=None) -> int:
    return _library().gemm_linear_act_grad(params, dy, lddy, pre, offsets, dz, lddz, dbias,
                                           workspace, workspace_bytes, stream)


def gemm_linear_weight_grad_workspace_size(params) -> int:
    return _library().gemm_linear_weight_grad_workspace_size(params)


def gemm_linear_weight_grad(params, x, dz, offsets, dtype_dw, beta, dw, workspace,
                            workspace_bytes, stream=None) -> int:
    return _library().gemm_linear_weight_grad(params, x, dz, offsets, dtype_dw, beta, dw,
                                              workspace, workspace_bytes, stream)


def gemm_linear_grad_workspace_size(params, outputs, dx=1, dw=1, dbias=1) -> int:
    return _library().gemm_linear_grad_workspace_size(params, outputs, dx, dw, dbias)


def gemm_linear_grad(params, outputs, dy, x, w, offsets, pre, dx, dw, dbias, workspace,
                     workspace_bytes, stream=None) -> int:
    return _library().gemm_linear_grad(params, outputs, dy, x, w, offsets, pre, dx, dw, dbias,
                                       workspace, workspace_bytes, stream)


def gemm_linear_num_configs(dtype: int) -> int:
    return _library().gemm_linear_num_configs(dtype)


def gemm_linear_config_name(dtype: int, cfg: int):
    name = _library().gemm_linear_config_name(dtype, cfg)
    return name.decode() if name is not None else None


def gemm_linear_config_forms(dtype: int, cfg: int) -> int:
    return _library().gemm_linear_config_forms(dtype, cfg)


def gemm_linear_select_config(params, weight_grad: int = 0) -> int:
    return _library().gemm_linear_select_config(params, weight_grad)


def gemm_linear_force_config(cfg: int = -1, split_k: int = 0) -> int:
    return _library().gemm_linear_force_config(cfg, split_k)


# ---------------------------------------------------------- torch helpers --

def _torch():
    global torch, _CODES, _raw_stream
    if _CODES is None:
        import torch as t
        torch = t
        # torch's current stream as a handle, without making a Stream object
        _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream",
                              lambda index: t.cuda.current_stream(index).cuda_stream)
        _CODES = {t.float32: 0, t.bfloat16: 1}   # last: it tells other threads that the rest is there
    return torch


torch = None
_CODES = None
_raw_stream = None


def _code(dtype, what):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, not %s" % (what, dtype))
    return code


def _matrix(t, rows, cols, dtype, device, what):
    """Leading dimension of a rows x cols matrix of that type and device."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    if tuple(t.shape) != (rows, cols) or t.device != device:
        raise ValueError("%s must be (%d, %d) on %s, not %s on %s"
                         % (what, rows, cols, device, tuple(t.shape), t.device))
    return _pitch(t, rows, cols, what)


def _pitch(t, rows, cols, what):
    if rows * cols == 0:
        return max(cols, 1)     # nothing is read or written: any stride will do
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError("the rows of %s must be contiguous" % what)
    return t.stride(-2) if rows > 1 else cols


def _weights(w, groups, transb):
    """(K, N, leading dimension, stride between groups) of w."""
    a, b = w.shape[-2], w.shape[-1]
    ld = _pitch(w, a, b, "w")   # a matrix of one row has contiguous values too
    stride = 0
    if groups:
        stride = w.stride(0) if groups > 1 and a * b else a * ld
    return (b, a, max(ld, 1), stride) if transb else (a, b, max(ld, 1), stride)


class _Launch:
    """Device, stream and memory of one call: the library launches on the
    calling thread's current device.  Memory for a stream that is not torch's
    current one comes from that stream's pool: a block of the current stream's
    pool may have been freed while kernels queued there still use it."""
    __slots__ = ("device", "index", "stream", "side", "guard")

    def __init__(self, device, stream):
        self.device, self.index = device, device.index
        current = _raw_stream(self.index)
        self.stream = current if stream is None else stream
        self.side = None if self.stream == current else torch.cuda.ExternalStream(self.stream, device=device)
        self.guard = None
        if torch.cuda.current_device() != self.index:
            self.guard = torch.cuda.device(device)
            self.guard.__enter__()

    def done(self):
        if self.guard is not None:
            self.guard.__exit__(None, None, None)

    def _take(self, shape, dtype):
        if self.side is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.side):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def empty(self, shape, dtype):
        """An output, which the caller may go on to use on the current stream."""
        t = self._take(shape, dtype)
        if self.side is not None and t.numel():
            t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def scratch(self, need):
        """(tensor kept alive by the caller, pointer) of `need` bytes."""
        if need < 0:
            _status(need)
        if need == 0:
            return None, None
        t = self._take((need,), torch.uint8)
        return t, t.data_ptr()


# Parameter blocks by their values, so that a repeated call does not fill one
# again; and their workspace sizes.
_blocks: dict = {}


def _block(*values):
    found = _blocks.get(values)
    if found is None:
        if len(_blocks) >= 4096:
            _blocks.clear()
        found = _blocks[values] = LinearParams(*values)
    return found


def _outputs(dtype_dx, dtype_dw, beta, lddx, lddw, stride_dw):
    values = (dtype_dx, dtype_dw, beta, 0, lddx, lddw, stride_dw)
    found = _blocks.get(values)
    if found is None:
        if len(_blocks) >= 4096:
            _blocks.clear()
        found = _blocks[values] = LinearGradOutputs(*values)
    return found


def _inputs(x, w, offsets, groups, transb, what="x"):
    if x.dim() != 2 or w.dim() != (3 if groups else 2):
        raise ValueError("%s must be 2-D and w %s" % (what, "3-D (groups first)" if groups else "2-D"))
    device = x.device
    if device.type != "cuda":
        raise ValueError("%s must be a GPU tensor" % what)
    if w.device != device:
        raise ValueError("%s and w must be on the same GPU" % what)
    if groups and (offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.device != device or
                   offsets.shape[0] != groups + 1 or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 tensor of %d values on the same GPU"
                         % (groups + 1))
    if w.dtype != x.dtype:
        raise TypeError("%s and w must both be float32 or both bfloat16" % what)
    return device, _code(x.dtype, what)


def _activation(act):
    code = ACTIVATIONS.get("none" if act is None else act)
    if code is None:
        raise ValueError("act must be one of %s, not %r" % (", ".join(ACTIVATIONS), act))
    return code


def _forward(x, w, offsets, groups, bias, act, residual, alpha, transb, pre, out, out_dtype, stream):
    _torch()
    device, dtype = _inputs(x, w, offsets, groups, transb)
    act = _activation(act)
    rows, K = x.shape
    K2, N, ldw, stride_w = _weights(w, groups, transb)
    if K != K2:
        raise ValueError("inner dimensions differ: x is %dx%d, w takes %d inputs" % (rows, K, K2))
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    dtype_y = _code(out_dtype, "y")
    ldx = _pitch(x, rows, K, "x")
    ldr = _matrix(residual, rows, N, out_dtype, device, "residual") if residual is not None else 0
    ldp = _matrix(pre, rows, N, out_dtype, device, "pre") if pre is not None else 0
    dtype_bias = stride_bias = 0
    if bias is not None:
        dtype_bias = _code(bias.dtype, "bias")
        if tuple(bias.shape) != ((groups, N) if groups else (N,)) or bias.device != device or \
                (N > 1 and bias.stride(-1) != 1):
            raise ValueError("bias must be %s with contiguous rows on x's device"
                             % ((groups, N) if groups else (N,),))
        stride_bias = bias.stride(0) if groups > 1 and N else N
    if out is not None:
        ldy = _matrix(out, rows, N, out_dtype, device, "out")
    else:
        ldy = max(N, 1)
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.empty((rows, N), out_dtype)
        params = _block(dtype, dtype_y, dtype_bias, 1 if transb else 0, act, float(alpha), rows, N, K,
                        groups, ldx, ldw, ldy, ldr, ldp, stride_w, stride_bias)
        lib = _library()
        need = lib.gemm_linear_workspace_size(params)
        ws, ws_ptr = at.scratch(need)
        rc = lib.gemm_linear(params, x.data_ptr(), w.data_ptr(),
                             offsets.data_ptr() if groups else None,
                             bias.data_ptr() if bias is not None else None,
                             residual.data_ptr() if residual is not None else None,
                             pre.data_ptr() if pre is not None else None, out.data_ptr(), ws_ptr,
                             need, at.stream)
    finally:
        at.done()
    _status(rc)
    return out


def linear(x, w, bias=None, act="none", residual=None, *, alpha=1.0, transb=False, pre=None,
           out=None, out_dtype=None, stream=None):
    """y = act(alpha * x . w + bias) + residual for GPU tensors.

    x (M x K) and w (K x N, or N x K with ``transb``) are both float32 or both
    bfloat16 with contiguous rows.  ``bias`` (N; float32 or bfloat16) and
    ``residual`` (M x N, y's type) are optional; ``act`` is "none", "relu",
    "gelu", "gelu_tanh" or "silu".  ``pre`` (M x N, y's type) receives the value
    before the activation, which the backward pass (``linear_grad``; autograd sees
    none of this) needs.  y is float32 or
    bfloat16 (``out_dtype``, default float32), created when ``out`` is not
    given; ``residual`` may be ``out`` itself.  Runs on ``stream`` (a handle;
    default: torch's current stream) and returns without synchronising.  On
    another stream than the current one the inputs have to be ready there, and
    whoever uses the outputs elsewhere waits for that stream first."""
    return _forward(x, w, None, 0, bias, act, residual, alpha, transb, pre, out, out_dtype, stream)


def grouped_linear(x, w, offsets, bias=None, act="none", residual=None, *, alpha=1.0, transb=False,
                   pre=None, out=None, out_dtype=None, stream=None):
    """``linear`` grouped by expert: rows offsets[g] .. offsets[g+1]-1 of x take
    w[g] and bias[g].

    w is G x K x N (G x N x K with ``transb``), bias G x N, and ``offsets`` an
    int32 GPU tensor of G + 1 non-decreasing row numbers, read on the GPU only.
    Groups may be empty.  Rows before offsets[0] and from offsets[G] on are not
    written: they keep what ``out`` holds (nothing defined, when it is created
    here)."""
    if w.dim() != 3 or w.shape[0] < 1:
        raise ValueError("w must be 3-D with at least one group")
    return _forward(x, w, offsets, w.shape[0], bias, act, residual, alpha, transb, pre, out,
                    out_dtype, stream)


def _backward(dy, x, w, offsets, groups, act, pre, alpha, transb, out_dtype, need_dx, need_dw,
              need_dbias, dw, accumulate, stream):
    _torch()
    device, dtype = _inputs(x, w, offsets, groups, transb)
    act = _activation(act)
    rows, K = x.shape
    K2, N, ldw, stride_w = _weights(w, groups, transb)
    if K != K2:
        raise ValueError("inner dimensions differ: x is %dx%d, w takes %d inputs" % (rows, K, K2))
    if out_dtype is None:
        out_dtype = dw.dtype if dw is not None else torch.float32
    dtype_out = _code(out_dtype, "the gradients")
    lddy = _matrix(dy, rows, N, x.dtype, device, "dy")
    ldx = _pitch(x, rows, K, "x")
    ldp, dtype_pre = 0, 0
    if act:
        if pre is None:
            raise ValueError("the gradient through an activation needs pre, its input")
        dtype_pre = _code(pre.dtype, "pre")
        ldp = _matrix(pre, rows, N, pre.dtype, device, "pre")
    if accumulate and dw is None:
        raise ValueError("accumulate needs an existing dw")
    if dw is not None:
        if tuple(dw.shape) != tuple(w.shape) or dw.device != device:
            raise ValueError("dw must have w's shape, on x's device")
        dtype_dw = _code(dw.dtype, "dw")
        _, _, ld_dw, stride_dw = _weights(dw, groups, transb)
    else:
        dtype_dw = dtype_out
        ld_dw = max(w.shape[-1], 1)
        stride_dw = w.shape[-2] * w.shape[-1] if groups else 0
    at = _Launch(device, stream)
    try:
        dx = at.empty((rows, K), out_dtype) if need_dx else None
        dbias = at.empty((groups, N) if groups else (N,), torch.float32) if need_dbias else None
        if need_dw and dw is None:
            dw = at.empty(tuple(w.shape), out_dtype)
        elif not need_dw:
            dw = None
        params = _block(dtype, dtype_pre, 0, 1 if transb else 0, act, float(alpha), rows, N, K, groups,
                        ldx, ldw, lddy, 0, ldp, stride_w, 0)
        outputs = _outputs(dtype_out, dtype_dw, 1.0 if accumulate else 0.0, max(K, 1), ld_dw, stride_dw)
        lib = _library()
        need = lib.gemm_linear_grad_workspace_size(params, outputs, need_dx, need_dw, need_dbias)
        ws, ws_ptr = at.scratch(need)
        rc = lib.gemm_linear_grad(params, outputs, dy.data_ptr(), x.data_ptr(), w.data_ptr(),
                                  offsets.data_ptr() if groups else None,
                                  pre.data_ptr() if act else None,
                                  dx.data_ptr() if need_dx else None,
                                  dw.data_ptr() if need_dw else None,
                                  dbias.data_ptr() if need_dbias else None, ws_ptr, need, at.stream)
    finally:
        at.done()
    _status(rc)
    return dx, dw, dbias


def linear_grad(dy, x, w, act="none", pre=None, *, alpha=1.0, transb=False, out_dtype=None,
                need_dx=True, need_dw=True, need_dbias=True, dw=None, accumulate=False, stream=None):
    """(dx, dw, dbias) of ``linear`` for the gradient dy of y (M x N, x's type):

        dz = dy * act'(pre)    dx = alpha * dz . w^T    dw = alpha * x^T . dz
        dbias = sum of dz over the rows

    (the residual's gradient is dy itself).  ``pre`` is what the forward pass
    stored; not needed without an activation.  dx and dw are ``out_dtype``
    (default float32), dw in w's layout, dbias float32.  Between an activation
    and the two products dz is rounded once to x's type, the one that the matrix
    cores read it in; dbias sums the values before that.  Where that rounding of
    a bfloat16 layer is too coarse (it adds as much to the error of dx and dw as
    their own rounding to bfloat16), pass dy, x and w as float32: nothing is
    rounded on the way then, at the float32 products' rate, and the gradients can
    still be bfloat16 (``out_dtype``).  ``dw`` receives the weight gradient when given, added to what
    it holds with ``accumulate``.  What is not needed comes back as None.
    ``stream`` as in ``linear``."""
    return _backward(dy, x, w, None, 0, act, pre, alpha, transb, out_dtype, need_dx, need_dw,
                     need_dbias, dw, accumulate, stream)


def grouped_linear_grad(dy, x, w, offsets, act="none", pre=None, *, alpha=1.0, transb=False,
                        out_dtype=None, need_dx=True, need_dw=True, need_dbias=True, dw=None,
                        accumulate=False, stream=None):
    """``linear_grad`` of ``grouped_linear``: dw (G x ...) and dbias (G x N) sum
    over each group's rows (zeros for an empty group); rows of dx outside the
    groups are not written."""
    if w.dim() != 3 or w.shape[0] < 1:
        raise ValueError("w must be 3-D with at least one group")
    return _backward(dy, x, w, offsets, w.shape[0], act, pre, alpha, transb, out_dtype, need_dx,
                     need_dw, need_dbias, dw, accumulate, stream)
