"""The operators around the layer (include/nmoe.h): the block's residual RMS norm, its dense
products in bf16 and in 8 bits, the router's balance loss, and their gradients.

Argument checks and marshalling only, like the rest of the binding: every call runs this
library's kernels on the tensors' device, on ``stream`` (default: the device's current
stream), and its outputs and workspace are allocated on that stream. Gradients are calls of
their own, which take what the forward call gave; nothing is recorded for autograd.

A block's step around the expert-choice layer::

    n = rms_norm(x, w, residual=res)                 # n.y feeds the router and the experts
    scores, scores_t = router(n.y, W_r)
    loss, counts = balance_loss(scores, k=2)
    dlogits = balance_loss_backward(scores, counts, k=2, dtype=torch.bfloat16)
    dy, dW_r, _ = linear_backward(dlogits, n.y, W_r)
    dx, dw = rms_norm_backward(dy, n.h, n.rstd, w)

(E a multiple of 8: the products' row lengths are, and other router weights need padding), and
a dense product in 8 bits::

    q_w, w_scale = quantize_rows(W.t().contiguous())  # once
    n = rms_norm(x, w, residual=res, out="fp8")
    y = linear_fp8(n.q, n.scale, q_w, w_scale, bias, act="gelu_tanh")
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._lib import SCORE, _check, _dt, _ptr, lib

ACT = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}
E4M3 = torch.float8_e4m3fn


class NormOut(NamedTuple):
    """What ``rms_norm`` gives: y and / or (q, scale) as asked for (else None), h = x +
    residual (x itself without a residual) and rstd, which the gradient takes."""
    y: Optional[torch.Tensor]
    h: torch.Tensor
    q: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    rstd: torch.Tensor


_device = torch._C._cuda_getDevice                    # the current device's index
# the current stream's handle as an int, without the Stream object that
# torch.cuda.current_stream() builds (3 us of a call that takes 10)
_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(fn, stream, *args):
    """Runs ``fn(*args)`` with its first argument's device and `stream` current, so that the
    call, its outputs and its workspace are all on that stream. Every call that is not on the
    current device's current stream comes through here."""
    t = args[0]
    if not t.is_cuda:
        raise ValueError(f"{fn.__name__}: the tensors must be CUDA tensors")
    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args)
        if stream.device != t.device:
            raise ValueError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on "
                             f"{t.device}")
        with torch.cuda.stream(stream):
            # an input that the caller drops must not be given out again before the stream
            # has read it
            for a in args:
                if isinstance(a, torch.Tensor):
                    a.record_stream(stream)
            return fn(*args)


def _need(t, name, device, shape, dtype):
    """Checks one tensor: device, dtype, shape, contiguous."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows(x, name):
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor")
    return x.shape


def _scratch(nbytes, device):
    """A workspace for one call (None if it needs none)."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def rms_norm(x, weight=None, residual=None, eps=1e-6, out="same", stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, over rows of x [T, d].

    ``out``: "same" gives y in x's dtype (bf16 or fp32), "fp8" gives q [T, d] e4m3 and
    scale [T] fp32 with y ~ q * scale, "both" gives both. Returns a NormOut."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(rms_norm, stream, x, weight, residual, eps, out)
    T, d = _rows(x, "x")
    dt = _dt(x)
    if out not in ("same", "fp8", "both"):
        raise ValueError(f"out must be 'same', 'fp8' or 'both', not {out!r}")
    if weight is not None:
        _need(weight, "weight", dev, (d,), x.dtype)
    h = None
    if residual is not None:
        _need(residual, "residual", dev, x.shape, x.dtype)
        h = torch.empty_like(x)
    y = torch.empty_like(x) if out != "fp8" else None
    q = scale = None
    if out != "same":
        q = torch.empty(T, d, dtype=E4M3, device=x.device)
        scale = torch.empty(T, dtype=torch.float32, device=x.device)
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(lib().nmoe_rms_norm(x.data_ptr(), _ptr(residual), _ptr(weight), T, d, eps, dt,
                               _ptr(h), _ptr(y), _ptr(q), _ptr(scale), rstd.data_ptr(),
                               _stream(dev)), "nmoe_rms_norm")
    return NormOut(y, x if h is None else h, q, scale, rstd)


def rms_norm_backward(dy, h, rstd, weight=None, dh=None, need_dweight=True, stream=None):
    """(dx, dweight fp32) from dy = the gradient of y, h and rstd as ``rms_norm`` gave them;
    ``dh`` is the gradient that reaches h from elsewhere. dx is the gradient of x and of
    the residual alike."""
    dev = dy.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(rms_norm_backward, stream, dy, h, rstd, weight, dh, need_dweight)
    T, d = _rows(dy, "dy")
    dt = _dt(dy)
    _need(h, "h", dev, dy.shape, dy.dtype)
    _need(rstd, "rstd", dev, (T,), torch.float32)
    if weight is not None:
        _need(weight, "weight", dev, (d,), dy.dtype)
    if dh is not None:
        _need(dh, "dh", dev, dy.shape, dy.dtype)
    dx = torch.empty_like(dy)
    dw = ws = None
    n = 0
    if need_dweight:
        dw = torch.empty(d, dtype=torch.float32, device=dy.device)
        n = lib().nmoe_rms_norm_backward_workspace(T, d)
        ws = _scratch(n, dy.device)
    _check(lib().nmoe_rms_norm_backward(dy.data_ptr(), h.data_ptr(), rstd.data_ptr(),
                                        _ptr(weight), _ptr(dh), T, d, dt, dx.data_ptr(),
                                        _ptr(dw), _ptr(ws), n, _stream(dev)),
           "nmoe_rms_norm_backward")
    return dx, dw


def quantize_rows(x, stream=None):
    """(q e4m3 [T, d], scale fp32 [T]) of the rows of x [T, d]: x ~ q * scale. Of W.t(), made
    contiguous, it is the weight of ``linear_fp8``."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(quantize_rows, stream, x)
    T, d = _rows(x, "x")
    q = torch.empty(T, d, dtype=E4M3, device=x.device)
    scale = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(lib().nmoe_quantize_rows(x.data_ptr(), T, d, _dt(x), q.data_ptr(), scale.data_ptr(),
                                    _stream(dev)), "nmoe_quantize_rows")
    return q, scale


def _out(out, M, N, out_f32, like, dev):
    dtype = torch.float32 if out_f32 else torch.bfloat16
    if out is None:
        return torch.empty(M, N, dtype=dtype, device=like.device)
    _need(out, "out", dev, (M, N), dtype)
    return out


def _epilogue_args(dev, bias, residual, M, N, act):
    if act not in ACT:
        raise ValueError(f"act must be one of {', '.join(ACT)}, not {act!r}")
    if bias is not None:
        _need(bias, "bias", dev, (N,), torch.bfloat16)
    if residual is not None:
        _need(residual, "residual", dev, (M, N), torch.bfloat16)


def linear(x, W, bias=None, act="none", residual=None, out_f32=False, preact=False, out=None,
           stream=None):
    """act(x W + bias) + residual, x [M, K], W [K, N], bias [N], residual [M, N] bf16.

    ``act``: "none", "silu", "gelu" or "gelu_tanh". Returns out [M, N] in bf16 (fp32 with
    ``out_f32``), or with ``preact`` the pair (out, x W + bias in bf16), whose second is
    what ``linear_backward`` needs of an activation. K and N are multiples of 8."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(linear, stream, x, W, bias, act, residual, out_f32, preact, out)
    M, K = _rows(x, "x")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x must be torch.bfloat16, not {x.dtype}")
    if W.dim() != 2:
        raise ValueError("W must be [K, N]")
    N = W.shape[1]
    _need(W, "W", dev, (K, N), torch.bfloat16)
    _epilogue_args(dev, bias, residual, M, N, act)
    out = _out(out, M, N, out_f32, x, dev)
    pre = torch.empty(M, N, dtype=torch.bfloat16, device=x.device) if preact else None
    _check(lib().nmoe_linear(x.data_ptr(), W.data_ptr(), _ptr(bias), _ptr(residual), M, K, N,
                             ACT[act], 1 if out_f32 else 0, _ptr(pre), out.data_ptr(),
                             _stream(dev)), "nmoe_linear")
    return (out, pre) if preact else out


def linear_fp8(q_x, x_scale, q_w, w_scale, bias=None, act="none", residual=None, out_f32=False,
               out=None, stream=None):
    """act((q_x * x_scale) (q_w * w_scale)^T + bias) + residual: q_x [M, K] and q_w [N, K]
    e4m3 with one fp32 scale a row each (from ``rms_norm`` and ``quantize_rows``), bias [N]
    and residual [M, N] bf16. Returns out [M, N] in bf16, or fp32 with ``out_f32``. K is a
    multiple of 16, N of 8."""
    dev = q_x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(linear_fp8, stream, q_x, x_scale, q_w, w_scale, bias, act, residual,
                          out_f32, out)
    M, K = _rows(q_x, "q_x")
    if q_x.dtype != E4M3:
        raise TypeError(f"q_x must be {E4M3}, not {q_x.dtype}")
    if q_w.dim() != 2:
        raise ValueError("q_w must be [N, K]")
    N = q_w.shape[0]
    _need(q_w, "q_w", dev, (N, K), E4M3)
    _need(x_scale, "x_scale", dev, (M,), torch.float32)
    _need(w_scale, "w_scale", dev, (N,), torch.float32)
    _epilogue_args(dev, bias, residual, M, N, act)
    out = _out(out, M, N, out_f32, q_x, dev)
    _check(lib().nmoe_linear_fp8(q_x.data_ptr(), x_scale.data_ptr(), q_w.data_ptr(),
                                 w_scale.data_ptr(), _ptr(bias), _ptr(residual), M, K, N,
                                 ACT[act], 1 if out_f32 else 0, out.data_ptr(),
                                 _stream(dev)), "nmoe_linear_fp8")
    return out


def linear_backward(dy, x, W, act="none", preact=None, need_dx=True, need_dW=True,
                    need_dbias=True, stream=None):
    """(dx [M, K] bf16, dW [K, N] bf16, dbias [N] fp32) of ``linear`` from dy [M, N] bf16
    (which is also the residual's gradient); the ones not needed are None. ``preact`` is
    what ``linear`` gave, with an activation; without one it is None. K and N are multiples of
    8, M is any."""
    dev = dy.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(linear_backward, stream, dy, x, W, act, preact, need_dx, need_dW,
                          need_dbias)
    M, N = _rows(dy, "dy")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    K = x.shape[1]
    bf = torch.bfloat16
    if dy.dtype != bf:
        raise TypeError(f"dy must be {bf}, not {dy.dtype}")
    _need(x, "x", dev, (M, K), bf)
    _need(W, "W", dev, (K, N), bf)
    if act not in ACT:
        raise ValueError(f"act must be one of {', '.join(ACT)}, not {act!r}")
    if (act != "none") != (preact is not None):
        raise ValueError("preact is needed with an activation, and only then")
    if preact is not None:
        _need(preact, "preact", dev, (M, N), bf)
    if not (need_dx or need_dW or need_dbias):
        raise ValueError("no gradient asked for")
    dx = torch.empty_like(x) if need_dx else None
    dW = torch.empty_like(W) if need_dW else None
    db = torch.empty(N, dtype=torch.float32, device=dy.device) if need_dbias else None
    n = lib().nmoe_linear_backward_workspace(M, K, N, ACT[act])
    ws = _scratch(n, dy.device)
    _check(lib().nmoe_linear_backward(dy.data_ptr(), x.data_ptr(), W.data_ptr(), _ptr(preact),
                                      M, K, N, ACT[act], _ptr(dx), _ptr(dW), _ptr(db),
                                      _ptr(ws), n, _stream(dev)), "nmoe_linear_backward")
    return dx, dW, db


def _balance_args(scores, mask, dev):
    T, E = _rows(scores, "scores")
    if scores.dtype != torch.float32:
        raise TypeError(f"scores must be torch.float32, not {scores.dtype}")
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"mask must be torch.bool or torch.uint8, not {mask.dtype}")
        _need(mask, "mask", dev, (T,), mask.dtype)
    return T, E


def balance_loss(scores, k: int, mask=None, n_segments=1, coef=1.0, stream=None):
    """(loss [n_segments] fp32, counts [n_segments, E] int32) of router scores [T, E]:
    coef * E * sum_e f_e P_e, f_e the share of expert e in the tokens' k best experts (ties
    to the lower expert) and P_e its mean score, over the tokens whose ``mask`` (bool or
    uint8 [T]) is set, each of the n_segments groups of T / n_segments tokens apart."""
    dev = scores.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(balance_loss, stream, scores, k, mask, n_segments, coef)
    T, E = _balance_args(scores, mask, dev)
    counts = torch.empty(n_segments, E, dtype=torch.int32, device=scores.device)
    loss = torch.empty(n_segments, dtype=torch.float32, device=scores.device)
    n = lib().nmoe_balance_loss_workspace(T, E, n_segments)
    ws = _scratch(n, scores.device)
    _check(lib().nmoe_balance_loss(scores.data_ptr(), _ptr(mask), T, E, k, n_segments, coef,
                                   counts.data_ptr(), loss.data_ptr(), _ptr(ws), n,
                                   _stream(dev)), "nmoe_balance_loss")
    return loss, counts


def balance_loss_backward(scores, counts, k: int, dloss=None, mask=None, n_segments=1, coef=1.0,
                          score_fn="softmax", dtype=torch.float32, stream=None):
    """The gradient of ``balance_loss`` with respect to the router's logits [T, E], in fp32 or
    bf16, through the score function the scores came from; counts as ``balance_loss`` gave
    them, dloss [n_segments] fp32 (None: ones)."""
    dev = scores.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(balance_loss_backward, stream, scores, counts, k, dloss, mask,
                          n_segments, coef, score_fn, dtype)
    T, E = _balance_args(scores, mask, dev)
    _need(counts, "counts", dev, (n_segments, E), torch.int32)
    if dloss is not None:
        _need(dloss, "dloss", dev, (n_segments,), torch.float32)
    if score_fn not in SCORE:
        raise ValueError(f"score_fn must be one of {', '.join(SCORE)}, not {score_fn!r}")
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype must be torch.float32 or torch.bfloat16, not {dtype}")
    d = torch.empty(T, E, dtype=dtype, device=scores.device)
    _check(lib().nmoe_balance_loss_backward(scores.data_ptr(), _ptr(mask), counts.data_ptr(),
                                            _ptr(dloss), T, E, k, n_segments, coef,
                                            SCORE[score_fn], _dt(d), d.data_ptr(),
                                            _stream(dev)), "nmoe_balance_loss_backward")
    return d
