"""What stands around a model's products when it answers, over torch tensors:
``moe_layer`` (a whole mixture-of-experts layer for a few tokens), ``adapter_linear``
(``linear`` with a low-rank adapter per row), ``log_probs`` (log probabilities of given
tokens, entropy, alternatives) and its gradient ``log_probs_grad``; a thin binding over
``include/gemm_serving.h``.  Like the rest of the package they take no part in torch's
autograd.  The C entry points are here under their own names (``gemm_*``), taking
parameters, device pointers and a stream."""
from __future__ import annotations

import collections
import ctypes

from . import layers
from .layers import _activation, _code, _i64, _int, _Launch, _library, _matrix, _p, _pitch, _status, _torch, _weights


class LogProbsParams(ctypes.Structure):
    """gemm_log_probs_params of include/gemm_serving.h."""
    _fields_ = [("dtype", ctypes.c_int32), ("top", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("ld", ctypes.c_int64)]


class MoeParams(ctypes.Structure):
    """gemm_moe_params of include/gemm_serving.h."""
    _fields_ = [(name, ctypes.c_int32) for name in ("dtype", "dtype_y", "transw", "act", "gated", "reserved")] + \
        [(name, ctypes.c_int64) for name in (
            "tokens", "hidden", "inner", "experts", "top", "ldx", "ldy", "ldr", "ldup", "lddown", "stride_up",
            "stride_down")]


class AdapterParams(ctypes.Structure):
    """gemm_adapter_params of include/gemm_serving.h."""
    _fields_ = [(name, ctypes.c_int32) for name in ("dtype", "dtype_y", "dtype_bias", "transw", "act", "reserved")] + \
        [(name, ctypes.c_int64) for name in (
            "rows", "N", "K", "adapters", "rank", "ldx", "ldw", "ldy", "ldr", "lda", "ldb", "stride_a", "stride_b")]


_plp = ctypes.POINTER(LogProbsParams)
_pmoe = ctypes.POINTER(MoeParams)
_pad = ctypes.POINTER(AdapterParams)
# Every symbol include/gemm_serving.h declares, with its ctypes signature.
SIGNATURES = {
    "gemm_moe_layer_workspace_size": (_i64, [_pmoe]),
    "gemm_moe_layer": (_int, [_pmoe] + [_p] * 8 + [_i64, _p]),
    "gemm_adapter_linear_workspace_size": (_i64, [_pad]),
    "gemm_adapter_linear": (_int, [_pad] + [_p] * 10 + [_i64, _p]),
    "gemm_log_probs_workspace_size": (_i64, [_plp]),
    "gemm_log_probs": (_int, [_plp] + [_p] * 8 + [_i64, _p]),
    "gemm_log_probs_grad": (_int, [_plp] + [_p] * 7 + [_i64, _p]),
}


# ---------------------------------------------------------------- C names --

def gemm_moe_layer_workspace_size(params) -> int:
    return _library().gemm_moe_layer_workspace_size(params)


def gemm_moe_layer(params, x, w_up, w_down, ids, weights, residual, y, workspace, workspace_bytes, stream=None) -> int:
    return _library().gemm_moe_layer(params, x, w_up, w_down, ids, weights, residual, y, workspace, workspace_bytes,
                                     stream)


def gemm_adapter_linear_workspace_size(params) -> int:
    return _library().gemm_adapter_linear_workspace_size(params)


def gemm_adapter_linear(params, x, w, a, b, ids, scales, bias, residual, y, workspace, workspace_bytes,
                        stream=None) -> int:
    return _library().gemm_adapter_linear(params, x, w, a, b, ids, scales, bias, residual, y, workspace,
                                          workspace_bytes, stream)


def gemm_log_probs_workspace_size(params) -> int:
    return _library().gemm_log_probs_workspace_size(params)


def gemm_log_probs(params, logits, tokens, logprob, entropy, stats, top_ids, top_logprobs, workspace,
                   workspace_bytes, stream=None) -> int:
    return _library().gemm_log_probs(params, logits, tokens, logprob, entropy, stats, top_ids, top_logprobs,
                                     workspace, workspace_bytes, stream)


def gemm_log_probs_grad(params, logits, tokens, stats, entropy, dlogprob, dentropy, dlogits, ldd,
                        stream=None) -> int:
    return _library().gemm_log_probs_grad(params, logits, tokens, stats, entropy, dlogprob, dentropy, dlogits, ldd,
                                          stream)


# ---------------------------------------------------------- torch helpers --

def _vector(t, shape, dtype, device, what):
    """Pointer of a contiguous tensor of that shape and type."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    if tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on %s, not %s on %s"
                         % (what, shape, device, tuple(t.shape), t.device))
    return t.data_ptr()


# Parameter blocks by their type and values, so that a repeated call does not
# fill one again.
_blocks: dict = {}


def _block(kind, *values):
    found = _blocks.get((kind, values))
    if found is None:
        if len(_blocks) >= 4096:
            _blocks.clear()
        found = _blocks[kind, values] = kind(*values)
    return found


def moe_layer(x, w_up, w_down, ids, weights, act="silu", residual=None, *, gated=True, transb=False, out=None,
              out_dtype=None, stream=None):
    """A whole mixture-of-experts layer for a few tokens (at most 512):

        h[t, j] = act(x_t . gate) * (x_t . up)   of expert ids[t, j]; act(x_t . up) without a gate
        y_t = sum_j weights[t, j] h[t, j] . down + residual_t

    x is tokens x hidden, ``ids`` (int32) and ``weights`` (float32) are contiguous,
    tokens x top, on the GPU and read there only.  ``w_up`` is experts x hidden x 2
    inner (the gate's columns first; inner without ``gated``), ``w_down`` experts x
    inner x hidden; with ``transb`` both are stored transposed.  x and the weights are
    all float32 or all bfloat16, with contiguous rows.  An id outside the experts counts
    for nothing.  y is ``out_dtype`` (default float32), created when ``out`` is not
    given; ``residual`` (y's type) may be ``out`` itself.  The router's part is
    ``log_probs``: its ``top_ids``, and the softmax of its ``top_logprobs``.  For long
    batches sort the rows by expert and use ``grouped_linear``, which reads the weights
    once for any number of rows.  ``stream`` as in ``linear``."""
    _torch()
    t = layers.torch
    if x.dim() != 2 or w_up.dim() != 3 or w_down.dim() != 3 or ids.dim() != 2:
        raise ValueError("x and ids must be 2-D, w_up and w_down 3-D (experts first)")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    if w_up.device != device or w_down.device != device:
        raise ValueError("x, w_up and w_down must be on the same GPU")
    if w_up.dtype != x.dtype or w_down.dtype != x.dtype:
        raise TypeError("x, w_up and w_down must all be float32 or all bfloat16")
    dtype, act = _code(x.dtype, "x"), _activation(act)
    tokens, hidden = x.shape
    experts, top = w_up.shape[0], ids.shape[1]
    hidden2, columns, ldup, stride_up = _weights(w_up, experts, transb)
    inner, hidden3, lddown, stride_down = _weights(w_down, experts, transb)
    if hidden2 != hidden or hidden3 != hidden or w_down.shape[0] != experts or columns != (2 * inner if gated else inner):
        raise ValueError("sizes differ: x is %dx%d, w_up %s, w_down %s" % (tokens, hidden, tuple(w_up.shape),
                                                                         tuple(w_down.shape)))
    ids_ptr = _vector(ids, (tokens, top), t.int32, device, "ids")
    weights_ptr = _vector(weights, (tokens, top), t.float32, device, "weights")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else t.float32
    dtype_y = _code(out_dtype, "y")
    ldr = _matrix(residual, tokens, hidden, out_dtype, device, "residual") if residual is not None else 0
    ldy = _matrix(out, tokens, hidden, out_dtype, device, "out") if out is not None else max(hidden, 1)
    params = _block(MoeParams, dtype, dtype_y, 1 if transb else 0, act, 1 if gated else 0, 0, tokens, hidden, inner,
                    experts, top, _pitch(x, tokens, hidden, "x"), ldy, ldr, ldup, lddown, stride_up, stride_down)
    at = _Launch(device, stream)
    try:
        lib = _library()
        need = lib.gemm_moe_layer_workspace_size(params)
        ws, ws_ptr = at.scratch(need)
        if out is None:
            out = at.empty((tokens, hidden), out_dtype)
        rc = lib.gemm_moe_layer(params, x.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), ids_ptr, weights_ptr,
                                residual.data_ptr() if residual is not None else None, out.data_ptr(), ws_ptr, need,
                                at.stream)
    finally:
        at.done()
    _status(rc)
    return out


def adapter_linear(x, w, a, b, ids, scales=None, bias=None, act="none", residual=None, *, transb=False, out=None,
                   out_dtype=None, stream=None):
    """``linear`` with a low-rank adapter per row, for the rows of many requests:

        y = act(x . w + bias + scales[i] (x . a[i]^T) . b[i]^T) + residual,  i = ids[row]

    x (M x K), w (K x N, or N x K with ``transb``), ``a`` (adapters x rank x K) and ``b``
    (adapters x N x rank) are all float32 or all bfloat16 with contiguous rows; ``ids``
    is a contiguous int32 tensor of M numbers on the GPU, read there only, in any order;
    one outside the adapters leaves its row without one.  ``scales`` (float32, one per
    adapter) is 1 if not given.  The rest as in ``linear``."""
    _torch()
    t = layers.torch
    if x.dim() != 2 or w.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x and w must be 2-D, a and b 3-D (adapters first)")
    device = x.device
    if device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    if w.device != device or a.device != device or b.device != device:
        raise ValueError("x, w, a and b must be on the same GPU")
    if w.dtype != x.dtype or a.dtype != x.dtype or b.dtype != x.dtype:
        raise TypeError("x, w, a and b must all be float32 or all bfloat16")
    dtype, act = _code(x.dtype, "x"), _activation(act)
    rows, K = x.shape
    K2, N, ldw, _ = _weights(w, 0, transb)
    count, rank = a.shape[0], a.shape[1]
    if K2 != K or tuple(a.shape) != (count, rank, K) or tuple(b.shape) != (count, N, rank):
        raise ValueError("sizes differ: x is %dx%d, w takes %d inputs to %d, a is %s, b is %s"
                         % (rows, K, K2, N, tuple(a.shape), tuple(b.shape)))
    _, _, lda, stride_a = _weights(a, count, False)
    _, _, ldb, stride_b = _weights(b, count, False)
    ids_ptr = _vector(ids, (rows,), t.int32, device, "ids")
    scales_ptr = _vector(scales, (count,), t.float32, device, "scales") if scales is not None else None
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else t.float32
    dtype_y = _code(out_dtype, "y")
    ldr = _matrix(residual, rows, N, out_dtype, device, "residual") if residual is not None else 0
    dtype_bias = 0
    if bias is not None:
        dtype_bias = _code(bias.dtype, "bias")
        _vector(bias, (N,), bias.dtype, device, "bias")
    ldy = _matrix(out, rows, N, out_dtype, device, "out") if out is not None else max(N, 1)
    params = _block(AdapterParams, dtype, dtype_y, dtype_bias, 1 if transb else 0, act, 0, rows, N, K, count, rank,
                    _pitch(x, rows, K, "x"), ldw, ldy, ldr, lda, ldb, stride_a, stride_b)
    at = _Launch(device, stream)
    try:
        lib = _library()
        need = lib.gemm_adapter_linear_workspace_size(params)
        ws, ws_ptr = at.scratch(need)
        if out is None:
            out = at.empty((rows, N), out_dtype)
        rc = lib.gemm_adapter_linear(params, x.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(), ids_ptr, scales_ptr,
                                     bias.data_ptr() if bias is not None else None,
                                     residual.data_ptr() if residual is not None else None, out.data_ptr(), ws_ptr,
                                     need, at.stream)
    finally:
        at.done()
    _status(rc)
    return out


def _logits(logits):
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be 2-D, rows x vocabulary")
    if logits.device.type != "cuda":
        raise ValueError("logits must be a GPU tensor")
    rows, vocab = logits.shape
    return _code(logits.dtype, "logits"), rows, vocab, _pitch(logits, rows, vocab, "logits")


LogProbs = collections.namedtuple("LogProbs", "logprob entropy stats top_ids top_logprobs")


def log_probs(logits, tokens=None, top=0, *, scale=1.0, stream=None):
    """Log probabilities of one token per row of logits, with the rows' entropy
    and most likely alternatives.

    ``logits`` (rows x vocabulary, float32 or bfloat16, contiguous rows) are
    multiplied by ``scale`` (1 / temperature, > 0, at most 2^64) first.  ``tokens`` is an int32
    tensor of one place per row; one outside the vocabulary is padding.  ``top`` (0
    to 64) alternatives come in falling order, equal logits by the lower place.
    Returns ``LogProbs``, float32 but for the places (int32):

        logprob        rows         of the token (0 for padding); None without tokens
        entropy        rows
        stats          rows x 2     the largest logit m, and log sum exp(scale (z - m)),
                                    which ``log_probs_grad`` takes
        top_ids        rows x top   None if top is 0
        top_logprobs   rows x top

    With a router's logits, ``top_ids`` are the experts and ``top_logprobs`` the
    logarithms of their shares, for ``moe_layer``.  -infinity is a forbidden place;
    NaN and +infinity make their row NaN.  Runs on ``stream`` (as in ``linear``) and
    returns without synchronising."""
    _torch()
    t = layers.torch
    dtype, rows, vocab, ld = _logits(logits)
    device = logits.device
    token_ptr = _vector(tokens, (rows,), t.int32, device, "tokens") if tokens is not None else None
    params = _block(LogProbsParams, dtype, top, float(scale), 0, rows, vocab, ld)
    lib = _library()
    need = lib.gemm_log_probs_workspace_size(params)
    if need < 0:
        raise ValueError("top must be 0 .. 64 and at most the vocabulary, scale positive and at most 2^64; not %r and %r"
                         % (top, scale))
    at = _Launch(device, stream)
    try:
        # one block for all of it, scratch included (at most some hundred KB): an
        # allocation takes the host 1.7 us, a view half of that
        held = rows if tokens is not None else 0
        fixed = (3 * rows + held + 2 * rows * top + 3) // 4 * 4
        block = at.empty((fixed + need // 4,), t.float32)
        base = block.data_ptr()
        stats, entropy = block.as_strided((rows, 2), (2, 1), 0), block.as_strided((rows,), (1,), 2 * rows)
        logprob = ids = alternatives = None
        if held:
            logprob = block.as_strided((rows,), (1,), 3 * rows)
        elif tokens is not None:
            logprob = block.as_strided((0,), (1,), 0)
        if top:
            first = 3 * rows + held
            alternatives = block.as_strided((rows, top), (top, 1), first)
            ids = block.view(t.int32).as_strided((rows, top), (top, 1), first + rows * top)
        at_top = base + 4 * (3 * rows + held)
        rc = lib.gemm_log_probs(params, logits.data_ptr(), token_ptr, base + 12 * rows if tokens is not None else None,
                                base + 8 * rows, base, at_top + 4 * rows * top if top else None,
                                at_top if top else None, base + 4 * fixed if need else None, need, at.stream)
    finally:
        at.done()
    _status(rc)
    return LogProbs(logprob, entropy, stats, ids, alternatives)


def log_probs_grad(logits, tokens, stats, entropy=None, dlogprob=None, dentropy=None, *, scale=1.0, out=None,
                   stream=None):
    """The gradient of sum(dlogprob * logprob + dentropy * entropy) with respect to
    the logits, in their type, from what ``log_probs`` returned for them (``stats``,
    and ``entropy`` where ``dentropy`` is given).

    ``dlogprob`` and ``dentropy`` are float32, one value per row; either may be
    left out.  Rows of padding tokens get zeros for the former.  ``out`` may be
    ``logits`` itself.  ``scale`` has to be the forward pass's."""
    _torch()
    t = layers.torch
    dtype, rows, vocab, ld = _logits(logits)
    device = logits.device
    stats_ptr = _vector(stats, (rows, 2), t.float32, device, "stats")
    token_ptr = _vector(tokens, (rows,), t.int32, device, "tokens") if tokens is not None else None
    entropy_ptr = _vector(entropy, (rows,), t.float32, device, "entropy") if entropy is not None else None
    dlogprob_ptr = _vector(dlogprob, (rows,), t.float32, device, "dlogprob") if dlogprob is not None else None
    dentropy_ptr = _vector(dentropy, (rows,), t.float32, device, "dentropy") if dentropy is not None else None
    if dlogprob is not None and tokens is None:
        raise ValueError("dlogprob needs tokens")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs entropy")
    params = _block(LogProbsParams, dtype, 0, float(scale), 0, rows, vocab, ld)
    ldd = _matrix(out, rows, vocab, logits.dtype, device, "out") if out is not None else vocab
    at = _Launch(device, stream)
    try:
        if out is None:
            out = at.empty((rows, vocab), logits.dtype)
        rc = _library().gemm_log_probs_grad(params, logits.data_ptr(), token_ptr, stats_ptr, entropy_ptr, dlogprob_ptr,
                                            dentropy_ptr, out.data_ptr(), ldd, at.stream)
    finally:
        at.done()
    _status(rc)
    return out
