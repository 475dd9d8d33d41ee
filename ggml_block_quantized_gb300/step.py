"""What stands around the products and the attention in a generation step: the
binding of include/qstep.h.

  norm_residual   adds a block's result to the residual stream, with a norm of it
                  and a gate where the model has them, and norms the sum for the
                  next block, in f32, f16 or the activation blocks qgemv_xq takes
  sample_tokens   the next tokens from the logits of the last product

As in the rest of the package, nothing here computes: tensors are checked,
outputs allocated with torch where none are passed, and the C entry points
called on the current stream (or `stream`).
"""
import ctypes

import torch

from .attention import _TYPE, _check, _new, _on, _place, _refuse, _stream

__all__ = ["norm_residual", "sample_tokens", "STEP_SYMBOLS"]

# every function declared in include/qstep.h
STEP_SYMBOLS = ("qnorm_residual", "qsample")

_F32 = (torch.float32,)


class _NormArgs(ctypes.Structure):
    """qnorm_args."""
    _fields_ = [("h", ctypes.c_void_p), ("y", ctypes.c_void_p), ("h_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("post_w", ctypes.c_void_p), ("post_b", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("w", ctypes.c_void_p), ("b", ctypes.c_void_p), ("h_out", ctypes.c_void_p),
                ("h_out_stride", ctypes.c_int64), ("x_out", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("d", ctypes.c_int64), ("h_type", ctypes.c_int32), ("y_type", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("act_type", ctypes.c_int32), ("layer", ctypes.c_int32), ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


_step = None


def _lib():
    """The loaded library with qstep.h's functions declared."""
    global _step
    if _step is None:
        from . import lib
        L = lib()
        i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        L.qnorm_residual.argtypes, L.qnorm_residual.restype = [ctypes.POINTER(_NormArgs), vp], i32
        L.qsample.argtypes = [i32, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.qsample.restype = i32
        _step = L
    return _step


def _matrix(t, device, name, dtypes, shape=None):
    """(address, stride from row to row) of a matrix whose rows are contiguous, of `shape` where it is given."""
    try:
        if t.dtype in dtypes and t.get_device() == device and t.dim() == 2 and (shape is None or t.shape == shape):
            if t.is_contiguous():
                return t.data_ptr(), t.shape[1]
            stride = t.stride()
            if stride[1] == 1 or t.shape[1] == 1:
                return t.data_ptr(), stride[0]
    except AttributeError:
        pass
    _refuse(t, device, name, dtypes)
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {list(shape) if shape is not None else '[rows, columns]'}, got {list(t.shape)}")
    raise ValueError(f"{name}: the elements of a row must be contiguous")


def _vector(t, device, name, n, dtype=torch.float32):
    """The address of t, contiguous [n]; None of None."""
    if t is None:
        return None
    at = _on(t, device, name, dtype)
    if t.shape != (n,):
        raise ValueError(f"{name} must be [{n}], got {list(t.shape)}")
    return at


# ------------------------------------------------------------ norms
def norm_residual(h, y=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale: float = 1.0,
                  eps: float = 1e-5, layer: bool = False, h_out=None, x_out=None, xq=None, act_type=None, stream=None):
    """h' = h + scale * gate * N(y; post_weight, post_bias) and x = N(h'; weight, bias) of the rows of h [n, d] and y
    [n, d] (float32 or float16 each). N divides by the root of the mean square plus eps, with `layer` after the mean was
    taken off; weights and biases are float32 [d] (None: 1 and none; y is taken as it is without post_weight). gate:
    float32 [d], or [n, d]. Without y, h' is h.

    Returns (h_out, x_out): h' in h's type (allocated where y is given and h_out is not; may be h itself) and x, in
    x_out's type (allocated in float32 if neither it nor xq is given; None where only xq is). xq: uint8, takes the rows of
    x as blocks of act_type (Q8_0, Q8_1, Q8_K), as quantize_act would make them, for qgemv_xq. x_out = False: no x."""
    device = _place(h, "h")
    h_ptr, h_stride = _matrix(h, device, "h", _TYPE)
    n, d = shape = h.shape
    y_ptr = y_stride = y_type = 0
    if y is not None:
        y_ptr, y_stride = _matrix(y, device, "y", _TYPE, shape)
        y_type = _TYPE[y.dtype]
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need y")
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias needs post_weight")
    if bias is not None and weight is None:
        raise ValueError("bias needs weight")
    gate_ptr, gate_stride = None, 0
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 1:
            gate_ptr = _vector(gate, device, "gate", d)
        else:
            gate_ptr, gate_stride = _matrix(gate, device, "gate", _F32, shape)
    h_out_ptr, h_out_stride = None, 0
    if h_out is None and y is not None:
        h_out = _new(shape, h.dtype, h.device, stream)
    if h_out is not None:
        h_out_ptr, h_out_stride = _matrix(h_out, device, "h_out", (h.dtype,), shape)
    xq_ptr = None
    if xq is not None:
        from . import Q8_0, Q8_1, Q8_K, qtype_nbytes
        if act_type not in (Q8_0, Q8_1, Q8_K):
            raise ValueError("xq needs act_type Q8_0, Q8_1 or Q8_K")
        need = qtype_nbytes(act_type, d)
        if need < 0:
            raise ValueError(f"rows of {d} are not whole blocks of act_type")
        xq_ptr = _on(xq, device, "xq", torch.uint8)
        if xq.numel() < n * need:
            raise ValueError(f"xq holds {xq.numel()} bytes, needs {n * need}")
    elif act_type is not None:
        raise ValueError("act_type without xq")
    x_ptr, x_type = None, 0
    if x_out is None and xq is None:
        x_out = _new(shape, torch.float32, h.device, stream)
    if x_out is not None and x_out is not False:
        x_ptr, x_stride = _matrix(x_out, device, "x_out", _TYPE, shape)
        if n > 1 and x_stride != d:
            raise ValueError("x_out must be contiguous")
        x_type = _TYPE[x_out.dtype]
    args = _NormArgs(h_ptr, y_ptr, h_stride, y_stride, _vector(post_weight, device, "post_weight", d),
                     _vector(post_bias, device, "post_bias", d), gate_ptr, gate_stride, _vector(weight, device, "weight", d),
                     _vector(bias, device, "bias", d), h_out_ptr, h_out_stride, x_ptr, xq_ptr, n, d, _TYPE[h.dtype], y_type,
                     x_type, act_type or 0, 1 if layer else 0, scale, eps)
    st = _lib().qnorm_residual(ctypes.byref(args), _stream(stream, device))
    if st:
        _check(st, "norm_residual")
    return h_out, None if x_out is False else x_out


# ------------------------------------------------------------ the next tokens
def sample_tokens(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, out=None, prob_out=None,
                  stream=None):
    """One token for each row of logits [n, vocab] (float32 or float16; rows may lie apart), int32 [n], and its
    probability among the tokens kept, float32 [n] (None unless prob_out is given). uniform: float32 [n], random numbers
    of [0, 1). temperature, top_p, min_p (float32 [n]) and top_k (int32 [n]) hold for each row by itself; None: 1 and
    all tokens. top_k keeps that many of the largest logits (0: all), top_p of those the likeliest until their share
    reaches it (1: all), min_p of those the ones at least that likely beside the likeliest; the likeliest always stays.
    Equal logits go by the lowest index. A temperature of 0 takes the largest logit; a row of -inf gives -1."""
    device = _place(logits, "logits")
    ptr, stride = _matrix(logits, device, "logits", _TYPE)
    n, vocab = logits.shape
    if uniform is None:
        raise TypeError("uniform must be a CUDA tensor")
    u_ptr = _vector(uniform, device, "uniform", n)
    t_ptr, p_ptr, m_ptr = (_vector(t, device, name, n) for t, name in
                           ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p")))
    k_ptr = _vector(top_k, device, "top_k", n, torch.int32)
    if out is None:
        out = _new((n,), torch.int32, logits.device, stream)
    out_ptr = _vector(out, device, "out", n, torch.int32)
    prob_ptr = _vector(prob_out, device, "prob_out", n)
    st = _lib().qsample(_TYPE[logits.dtype], ptr, stride, n, vocab, t_ptr, k_ptr, p_ptr, m_ptr, u_ptr, out_ptr, prob_ptr,
                        _stream(stream, device))
    if st:
        _check(st, "sample_tokens")
    return out, prob_out
