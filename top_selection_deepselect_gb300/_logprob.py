"""ctypes binding of include/ds_logprob.h -- log probabilities of given tokens,
entropy, the likeliest alternatives and their gradient -- argument marshalling
only, as in _binding.

The functions named like C entry points take the same arguments; token_logprobs
and token_logprobs_backward take torch tensors, allocate outputs with torch and
enqueue on the current stream of the tensors' device, which need not be the
current device.
"""
import ctypes

from . import _kv4
from ._binding import _check, load_library

LOGPROB_ENTRY_POINTS = ["ds_token_logprobs", "ds_token_logprobs_backward"]

_typed = None


def _lib():
    global _typed
    if _typed is None:
        lib = load_library()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        lib.ds_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, i32, f32, vp, vp, vp, vp, vp, vp]
        lib.ds_token_logprobs.restype = i32
        lib.ds_token_logprobs_backward.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, f32, vp, vp, vp, vp,
                                                   vp, vp, vp, i64, vp]
        lib.ds_token_logprobs_backward.restype = i32
        _typed = lib
    return _typed


# ---- C entry points, same names and argument order ---------------------------
def ds_token_logprobs(logits, dtype, rows, vocab, row_stride, tokens, k, scale, logprob, entropy, lse,
                      idx, top, stream):
    return _check(_lib().ds_token_logprobs(logits, dtype, rows, vocab, row_stride, tokens, k, scale,
                                           logprob, entropy, lse, idx, top, stream),
                  "ds_token_logprobs")


def ds_token_logprobs_backward(logits, dtype, rows, vocab, row_stride, tokens, k, idx, scale, lse,
                               entropy, grad_logprob, grad_entropy, grad_lse, grad_top, grad,
                               grad_stride, stream):
    return _check(_lib().ds_token_logprobs_backward(
        logits, dtype, rows, vocab, row_stride, tokens, k, idx, scale, lse, entropy, grad_logprob,
        grad_entropy, grad_lse, grad_top, grad, grad_stride, stream), "ds_token_logprobs_backward")


# ---- torch convenience wrappers ------------------------------------------------
_t = _kv4._t


def _logits(t, name, x, index):
    """(address, rows, vocab, row stride) of a [rows, vocab] tensor on device `index`."""
    if x.dim() != 2 or x.get_device() != index:
        raise ValueError("%s must be [rows, vocab] on cuda:%d" % (name, index))
    rows, vocab = x.shape
    stride, unit = x.stride()
    if unit != 1 and vocab != 1:
        raise ValueError("%s must have unit stride in the last dimension" % name)
    if stride < vocab:
        if rows > 1:
            raise ValueError("rows of %s must not overlap" % name)
        stride = vocab
    return x.data_ptr(), rows, vocab, stride


def _float32(t, name, x, shape, index):
    """Address of a contiguous float32 tensor of this shape on device `index`."""
    if x.dtype is not t.float32 or x.get_device() != index or x.shape != shape or not x.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of shape %s on cuda:%d"
                         % (name, tuple(shape), index))
    return x.data_ptr()


def token_logprobs(logits, tokens, k=0, scale=1.0, logprob=None, entropy=None, lse=None, idx=None,
                   top=None, stream=None):
    """Log probability of each row's given token, the row's entropy, and its k likeliest tokens.

    logits: [rows, vocab] float32, bfloat16 or float16, unit stride in the last
    dimension; the distribution is softmax(scale * logits).  tokens: int32
    [rows]; a token outside [0, vocab) (padding) has log probability 0.
    0 <= k <= 32.  Returns (logprob, entropy, lse) float32 [rows] and (idx int32,
    top float32) [rows, k]: the k first tokens by (logit descending, index
    ascending) and their log probabilities.

    Where logits requires a gradient, logprob, entropy, lse and top have one
    (outputs are then allocated, not given).  There is no forward-mode derivative:
    logits that carry a tangent are refused.
    """
    t = _t if _t.ready else _t.find()
    index = _kv4._cuda("logits", logits)
    if stream is not None or index != t.current():
        return _kv4._elsewhere(t, index, stream, token_logprobs,
                               logits, tokens, k, scale, logprob, entropy, lse, idx, top)
    if t.unpack_dual(logits).tangent is not None:
        raise NotImplementedError("token_logprobs has no forward-mode derivative")
    if logits.requires_grad and t.torch.is_grad_enabled():
        if any(x is not None for x in (logprob, entropy, lse, idx, top)):
            raise ValueError("outputs cannot be given where logits requires a gradient")
        return _function(t).apply(logits, tokens, k, scale)
    return _forward(t, index, logits, tokens, k, scale, logprob, entropy, lse, idx, top)


def _forward(t, index, logits, tokens, k, scale, logprob, entropy, lse, idx, top):
    code = t.codes.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be float32, bfloat16 or float16, got %s" % logits.dtype)
    at, rows, vocab, stride = _logits(t, "logits", logits, index)
    tokens_at = _kv4._int32("tokens", tokens, index, rows)
    device = logits.device
    if logprob is None:
        logprob = t.empty(rows, dtype=t.float32, device=device)
    else:
        _float32(t, "logprob", logprob, (rows,), index)
    if entropy is None:
        entropy = t.empty(rows, dtype=t.float32, device=device)
    else:
        _float32(t, "entropy", entropy, (rows,), index)
    if lse is None:
        lse = t.empty(rows, dtype=t.float32, device=device)
    else:
        _float32(t, "lse", lse, (rows,), index)
    width = k if k > 0 else 0
    if idx is None:
        idx = t.empty((rows, width), dtype=t.int32, device=device)
    elif idx.shape != (rows, width):
        raise ValueError("idx must have shape (%d, %d), got %s" % (rows, width, tuple(idx.shape)))
    else:
        _kv4._int32("idx", idx, index)
    if top is None:
        top = t.empty((rows, width), dtype=t.float32, device=device)
    else:
        _float32(t, "top", top, (rows, width), index)
    status = _lib().ds_token_logprobs(
        at, code, rows, vocab, stride, tokens_at, k, scale, logprob.data_ptr(), entropy.data_ptr(),
        lse.data_ptr(), idx.data_ptr(), top.data_ptr(), t.raw_stream(index))
    if status:
        _check(status, "ds_token_logprobs")
    return logprob, entropy, lse, idx, top


def token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob=None, grad_entropy=None,
                            idx=None, grad_top=None, grad_lse=None, scale=1.0, out=None, stream=None):
    """Gradient by the logits of what token_logprobs returned for the same logits, tokens and scale.

    lse and entropy (and idx, where grad_top is given) are that call's; a gradient
    that is None is 0.  Returns a tensor like logits; `out` may be logits itself.
    """
    t = _t if _t.ready else _t.find()
    index = _kv4._cuda("logits", logits)
    if stream is not None or index != t.current():
        return _kv4._elsewhere(t, index, stream, token_logprobs_backward, logits, tokens, lse, entropy,
                               grad_logprob, grad_entropy, idx, grad_top, grad_lse, scale, out)
    code = t.codes.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be float32, bfloat16 or float16, got %s" % logits.dtype)
    at, rows, vocab, stride = _logits(t, "logits", logits, index)
    if out is None:
        out = t.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    elif out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must have logits' shape and dtype")
    out_at, _, _, out_stride = _logits(t, "out", out, index)
    size = out.element_size()
    if out_at == at:
        if rows > 1 and out_stride != stride:
            raise ValueError("out may be logits itself, with the same strides, or apart from it")
    elif rows and out_at < at + ((rows - 1) * stride + vocab) * size and (
            at < out_at + ((rows - 1) * out_stride + vocab) * size) and not (
            _apart(at, out_at, stride, out_stride, rows, vocab, size)):
        raise ValueError("out may be logits itself, with the same strides, or apart from it")
    rows_of = (rows,)

    def given(name, x, shape=rows_of):
        return None if x is None else _float32(t, name, x, shape, index)

    k, idx_at = 0, None
    if grad_top is not None:
        if idx is None:
            raise ValueError("grad_top needs idx")
        if idx.dim() != 2 or idx.shape[0] != rows:
            raise ValueError("idx must be [rows, k]")
        k = idx.shape[1]
        idx_at = _kv4._int32("idx", idx, index)
    status = _lib().ds_token_logprobs_backward(
        at, code, rows, vocab, stride, _kv4._int32("tokens", tokens, index, rows), k, idx_at, scale,
        _float32(t, "lse", lse, rows_of, index), _float32(t, "entropy", entropy, rows_of, index),
        given("grad_logprob", grad_logprob), given("grad_entropy", grad_entropy),
        given("grad_lse", grad_lse), given("grad_top", grad_top, (rows, k)), out_at, out_stride,
        t.raw_stream(index))
    if status:
        _check(status, "ds_token_logprobs_backward")
    return out


def _apart(a, b, a_stride, b_stride, rows, vocab, size):
    """Whether rows of two tensors that lie in the same stretch of memory miss each other: columns
    of one wide tensor do."""
    if a_stride != b_stride:
        return False
    step = a_stride * size
    shift = (b - a) % step
    return vocab * size <= shift <= step - vocab * size


_made = None


def _function(t):
    """The autograd function, made at the first call that needs it."""
    global _made
    if _made is not None:
        return _made

    class TokenLogprobs(t.torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, tokens, k, scale):
            logprob, entropy, lse, idx, top = _forward(t, logits.get_device(), logits, tokens, k, scale,
                                                       None, None, None, None, None)
            ctx.save_for_backward(logits, tokens, lse, entropy, idx)
            ctx.scale = scale
            ctx.mark_non_differentiable(idx)
            ctx.set_materialize_grads(False)
            return logprob, entropy, lse, idx, top

        @staticmethod
        @t.torch.autograd.function.once_differentiable
        def backward(ctx, grad_logprob, grad_entropy, grad_lse, grad_idx, grad_top):
            logits, tokens, lse, entropy, idx = ctx.saved_tensors
            grads = [None if g is None else g.float().contiguous()
                     for g in (grad_logprob, grad_entropy, grad_lse, grad_top)]
            if all(g is None for g in grads):
                return None, None, None, None
            return token_logprobs_backward(logits, tokens, lse, entropy, grads[0], grads[1], idx, grads[3],
                                           grads[2], ctx.scale), None, None, None

    _made = TokenLogprobs
    return _made
