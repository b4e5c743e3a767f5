"""The operators around the grouped GEMM of a mixture-of-experts layer.

``gate_topk`` chooses each token's experts before ``route``, ``unroute`` brings the packed rows
back, ``silu_mul`` stands between the two expert products, ``pack8`` keeps rows in 8 bits; each
with its gradient, as thin calls of the C ABI that write into the caller's buffers (buffers left
as None are allocated, uninitialised, for the stream that the call runs on). ``gate``,
``dispatch``, ``swiglu``, ``expert_mlp`` and ``combine`` are the same operators with autograd, to
stand beside ``grouped_mm``; they run on the current stream, their backward passes do not support
being differentiated again, and tensors with a tangent (forward-mode differentiation) are refused.

Capture in a CUDA graph: the calls that write into buffers need nothing but their buffers. A
backward pass of the autograd forms can be captured like any other of torch: together with its
forward pass, and while no eager graph of the same leaves lives (torch ties a leaf's gradient to
the stream of the graph that used it first, and a capture cannot wait for that stream).
"""
from __future__ import annotations

import ctypes
import importlib
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (FLAG_GATE_UP_CONCAT, FLAG_ZERO_TAIL, _check, _raise, _status_ptr, _stream_handle,
               _wants_grad, dgrad_ex, forward_ex, lib, route, wgrad_ex)
from ._native_name import native_name


def _load_native():
    """csrc/binding.cpp: the calls below with their buffers in hand, 3 us sooner. None where it is
    not built for this interpreter and this torch: the same through ctypes."""
    try:
        return importlib.import_module("." + native_name(), __package__)
    except ImportError:
        return None


_native = _load_native()

GATE_SOFTMAX, GATE_SIGMOID = 0, 1
GATE_RENORM, GATE_LOGITS_F32 = 0x1, 0x2
GATE_MAX_K = 32
BLOCK8 = 32  # columns that share a scale of the 8-bit row form

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def declare(L: ctypes.CDLL) -> None:
    """Argument types of this module's entry points."""
    global _native
    if _native is None:  # built since this module was imported
        _native = _load_native()
    P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    for name, args in {
        "gg_gate_topk": [P, i64, i32, i32, P, i32, i32, f32, P, P, P, P, P],
        "gg_gate_topk_backward": [P, i64, i32, i32, i32, i32, f32, P, P, P, P, P],
        "gg_unroute": [P, i64, P, P, P, i64, i32, i64, P, P, P],
        "gg_unroute_backward": [P, P, i64, P, P, i64, i32, i64, P, i32, P, P, P, P],
        "gg_silu_mul": [P, i64, i64, P, P, i64, P, i32, P, P, P, P, P],
        "gg_silu_mul_backward": [P, P, P, P, i64, i64, P, P, i64, P, i32, P, P, P, P, P],
        "gg_pack8": [P, i64, i64, P, P, P, P, P],
        "gg_unpack8": [P, P, i64, i64, P, i32, P, P, P],
    }.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
        if _native is not None:
            _native.bind(name, ctypes.cast(fn, P).value)


def _on(stream):
    """Allocate for the stream that the call runs on, not for the current one."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _arg(t, name, shape, dtype, dev) -> Optional[int]:
    """Address of an argument of this shape and type (None: NULL) on device ``dev``, the current
    one. One combined test for the usual case, the messages of ``_check`` for the others."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    _check(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _new(t, shape, dtype, like, stream):
    """The caller's buffer, or a new one."""
    if t is not None:
        return t
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _vector(t, name, dtype, dev):
    """(address, entries) of a one-dimensional argument of any length."""
    n = t.numel() if isinstance(t, torch.Tensor) else 0
    return _arg(t, name, (n,), dtype, dev), n


def _used_ptr(offs, zero_tail, dev):
    """Address of the last offset: the number of packed rows in use."""
    if offs is None:
        if zero_tail:
            raise ValueError("zero_tail needs offs")
        return None
    p, n = _vector(offs, "offs", _I32, dev)
    if n == 0:
        raise ValueError("offs must not be empty")
    return p + 4 * (n - 1)


# ------------------------------------------------------------------------------------- gate

def _gate_args(logits, k, score, renorm, scale):
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (_BF16, _F32):
        raise TypeError("logits must be a torch.bfloat16 or torch.float32 tensor")
    _check(logits, "logits", logits.dtype, 2)
    if score not in (GATE_SOFTMAX, GATE_SIGMOID):
        raise ValueError("score must be GATE_SOFTMAX or GATE_SIGMOID")
    flags = (GATE_RENORM if renorm else 0) | (GATE_LOGITS_F32 if logits.dtype is _F32 else 0)
    T, E = logits.shape
    return T, E, int(k), int(score), flags, float(scale), logits.get_device()


def gate_topk(logits: torch.Tensor, k: int, *, score: int = GATE_SOFTMAX, renorm: bool = True,
              scale: float = 1.0, bias: Optional[torch.Tensor] = None,
              num_tokens: Optional[torch.Tensor] = None,
              topk_ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None):
    """Each token's k experts and their weights. Returns (topk_ids int32 [T, k], weights
    float32 [T, k]), best first, ties to the lowest expert.

    logits bf16 or float32 [T, E]; weights are scale * softmax(logits) (or the sigmoid) of the
    chosen experts, divided by their sum with ``renorm``. ``bias`` float32 [E]
    (GATE_SIGMOID only) is added to the scores for the choice alone. Logits of -inf are masked;
    a token with fewer than k others gets ids -1, which ``route`` drops, and weights 0 in its
    last slots. ``num_tokens`` int32 [1]: tokens in use of a padded batch, read on the device."""
    if _native is not None:
        rc = _native.gate_topk(logits, k, score, renorm, scale, bias, num_tokens, topk_ids,
                               weights, status, stream)
        if rc is not None:
            _raise(rc, "gg_gate_topk")
            return topk_ids, weights
    T, E, k, score, flags, scale, dev = _gate_args(logits, k, score, renorm, scale)
    if k < 1:
        raise ValueError("k must be positive")
    ids = _new(topk_ids, (T, k), _I32, logits, stream)
    w = _new(weights, (T, k), _F32, logits, stream)
    rc = lib().gg_gate_topk(
        logits.data_ptr(), T, E, k, _arg(bias, "bias", (E,), _F32, dev), score, flags, scale,
        _arg(num_tokens, "num_tokens", (1,), _I32, dev), _arg(ids, "topk_ids", (T, k), _I32, dev),
        _arg(w, "weights", (T, k), _F32, dev), _status_ptr(status), _stream_handle(stream, dev))
    _raise(rc, "gg_gate_topk")
    return ids, w


def gate_topk_backward(logits: torch.Tensor, topk_ids: torch.Tensor, dweights: torch.Tensor,
                       dlogits: Optional[torch.Tensor] = None, *, score: int = GATE_SOFTMAX,
                       renorm: bool = True, scale: float = 1.0,
                       status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the logits (in their type, written in full) from that of the weights;
    ``topk_ids`` is what ``gate_topk`` returned for the same score, renorm and scale. Not in place:
    ``dlogits`` must not overlap the logits."""
    if _native is not None:
        rc = _native.gate_topk_backward(logits, topk_ids, dweights, dlogits, score, renorm, scale,
                                        status, stream)
        if rc is not None:
            _raise(rc, "gg_gate_topk_backward")
            return dlogits
    _check(topk_ids, "topk_ids", _I32, 2)
    T, E, k, score, flags, scale, dev = _gate_args(logits, topk_ids.shape[1], score, renorm,
                                                   scale)
    if topk_ids.shape[0] != T:
        raise ValueError("topk_ids[T, k] and logits[T, E] disagree on T")
    out = _new(dlogits, (T, E), logits.dtype, logits, stream)
    rc = lib().gg_gate_topk_backward(
        logits.data_ptr(), T, E, k, score, flags, scale, topk_ids.data_ptr(),
        _arg(dweights, "dweights", (T, k), _F32, dev),
        _arg(out, "dlogits", (T, E), logits.dtype, dev), _status_ptr(status),
        _stream_handle(stream, dev))
    _raise(rc, "gg_gate_topk_backward")
    return out


# ---------------------------------------------------------------------------------- unroute

def _tokens(row_of, k, dev):
    """(tokens, k, address) of row_of."""
    rp, n = _vector(row_of, "row_of", _I32, dev)
    k = int(k)
    if rp is None or k < 1 or n % k != 0:
        raise ValueError("row_of must hold k entries for each token")
    return n // k, k, rp


def unroute(Y: torch.Tensor, row_of: torch.Tensor, k: int, out: Optional[torch.Tensor] = None, *,
            weights: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t,:] = residual[t,:] + sum over a token's k slots of weights[t,s] * Y[row_of[t*k+s],:],
    summed in fp32 in the order of the slots.

    Y bf16 [rows, N]; row_of int32 [T*k] from ``route`` (-1 adds nothing); weights float32 [T, k]
    (None: 1); residual bf16 [T, N] (None: 0; may be ``out``); out bf16 [T, N]."""
    if _native is not None:
        rc = _native.unroute(Y, row_of, k, out, weights, residual, status, stream)
        if rc is not None:
            _raise(rc, "gg_unroute")
            return out
    _check(Y, "Y", _BF16, 2)
    dev = Y.get_device()
    T, k, rp = _tokens(row_of, k, dev)
    rows, N = Y.shape
    out = _new(out, (T, N), _BF16, Y, stream)
    rc = lib().gg_unroute(Y.data_ptr(), rows, rp, _arg(weights, "weights", (T, k), _F32, dev),
                          _arg(residual, "residual", (T, N), _BF16, dev), T, k, N,
                          _arg(out, "out", (T, N), _BF16, dev), _status_ptr(status),
                          _stream_handle(stream, dev))
    _raise(rc, "gg_unroute")
    return out


def unroute_backward(dout: torch.Tensor, row_of: torch.Tensor, k: int,
                     dY: Optional[torch.Tensor] = None, *, Y: Optional[torch.Tensor] = None,
                     weights: Optional[torch.Tensor] = None,
                     dweights: Optional[torch.Tensor] = None,
                     offs: Optional[torch.Tensor] = None, zero_tail: bool = False,
                     status: Optional[torch.Tensor] = None, stream=None):
    """Gradients of ``unroute`` into the caller's buffers, either of which may be None: dY bf16
    [rows, N] (row row_of[i] becomes weights[i] * dout of its token) and dweights float32 [T, k]
    (needs Y). Rows of dY that row_of does not name are left as they are; with ``zero_tail``
    those past the last of ``offs`` become zeros. row_of's rows must be distinct. Returns
    (dY, dweights)."""
    if _native is not None:
        rc = _native.unroute_backward(dout, row_of, k, dY, Y, weights, dweights, offs, zero_tail,
                                      status, stream)
        if rc is not None:
            _raise(rc, "gg_unroute_backward")
            return dY, dweights
    _check(dout, "dout", _BF16, 2)
    dev = dout.get_device()
    T, k, rp = _tokens(row_of, k, dev)
    N = dout.shape[1]
    if dout.shape[0] != T:
        raise ValueError("dout must have a row for each token")
    if dY is None and dweights is None:
        raise ValueError("one of dY and dweights must be given")
    if dweights is not None and Y is None:
        raise ValueError("dweights needs Y")
    packed, name = (dY, "dY") if dY is not None else (Y, "Y")
    _check(packed, name, _BF16, 2)
    rows = packed.shape[0]
    rc = lib().gg_unroute_backward(
        dout.data_ptr(), _arg(Y, "Y", (rows, N), _BF16, dev), rows, rp,
        _arg(weights, "weights", (T, k), _F32, dev), T, k, N, _used_ptr(offs, zero_tail, dev),
        FLAG_ZERO_TAIL if zero_tail else 0, _arg(dY, "dY", (rows, N), _BF16, dev),
        _arg(dweights, "dweights", (T, k), _F32, dev), _status_ptr(status),
        _stream_handle(stream, dev))
    _raise(rc, "gg_unroute_backward")
    return dY, dweights


# --------------------------------------------------------------- SiLU-and-mul, 8-bit rows

def _half_blocks(N):
    return 2 * ((N // 2 + BLOCK8 - 1) // BLOCK8)


def _act_args(first, offs, row_of, weights, gate_up_concat, zero_tail, dev):
    """(rows_used, row_of, n_assign, weights, flags): pointers and sizes of the C call, whose
    first argument is the rows ``first``."""
    used = _used_ptr(offs, zero_tail, dev)
    n, rp, na = first.shape[0], None, 0
    if row_of is not None:
        rp, na = _vector(row_of, "row_of", _I32, dev)
        rp = rp or first.data_ptr()  # of no assignment: not NULL, not read
        n = na
    return (used, rp, na, _per_row(weights, "weights", n, dev),
            (FLAG_ZERO_TAIL if zero_tail else 0) | (FLAG_GATE_UP_CONCAT if gate_up_concat else 0))


def _per_row(t, name, n, dev):
    """float32, one for each assignment (of any shape, e.g. [T, k]) or row."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values")
    return _arg(t, name, t.shape, _F32, dev)


def _args8(x8, scale, rows, cols, codes, dev):
    """Addresses of the 8-bit rows and their scales."""
    if (x8 is None) != (scale is None):
        raise ValueError("H8 and H8_scale go together")
    return (_arg(x8, "H8", (rows, cols), _E4M3, dev),
            _arg(scale, "H8_scale", (rows, codes), _E8M0, dev))


def silu_mul(H: torch.Tensor, act: Optional[torch.Tensor] = None, *,
             offs: Optional[torch.Tensor] = None, row_of: Optional[torch.Tensor] = None,
             weights: Optional[torch.Tensor] = None, gate_up_concat: bool = False,
             zero_tail: bool = False, H8: Optional[torch.Tensor] = None,
             H8_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """act[r,:] = weight * silu(gate) * up of the packed rows H bf16 [rows, N]; act bf16
    [rows, N/2]. Gate and up columns lie in blocks of 128 in turn (N % 256 == 0) or, with
    ``gate_up_concat``, as the halves of N (N % 16 == 0).

    Rows are those before the last of ``offs`` (None: all), with weights[r]; or, with ``row_of``
    from ``route``, the rows that it names, with weights[i] of assignment i (any shape). With
    ``H8`` float8_e4m3fn [rows, N] and ``H8_scale`` float8_e8m0fnu [rows, 2*ceil(N/64)] the rows
    of H are also kept there in 8 bits, for ``silu_mul_backward``."""
    if _native is not None:
        rc = _native.silu_mul(H, act, offs, row_of, weights, gate_up_concat, zero_tail, H8,
                              H8_scale, status, stream)
        if rc is not None:
            _raise(rc, "gg_silu_mul")
            return act
    _check(H, "H", _BF16, 2)
    rows, N = H.shape
    dev = H.get_device()
    used, rp, n, wp, flags = _act_args(H, offs, row_of, weights, gate_up_concat, zero_tail, dev)
    p8, ps = _args8(H8, H8_scale, rows, N, _half_blocks(N), dev)
    act = _new(act, (rows, N // 2), _BF16, H, stream)
    rc = lib().gg_silu_mul(H.data_ptr(), rows, N, used, rp, n, wp, flags,
                           _arg(act, "act", (rows, N // 2), _BF16, dev), p8, ps,
                           _status_ptr(status), _stream_handle(stream, dev))
    _raise(rc, "gg_silu_mul")
    return act


def silu_mul_backward(dact: torch.Tensor, dH: Optional[torch.Tensor] = None, *,
                      H: Optional[torch.Tensor] = None, H8: Optional[torch.Tensor] = None,
                      H8_scale: Optional[torch.Tensor] = None,
                      offs: Optional[torch.Tensor] = None,
                      row_of: Optional[torch.Tensor] = None,
                      weights: Optional[torch.Tensor] = None,
                      act: Optional[torch.Tensor] = None,
                      dweights: Optional[torch.Tensor] = None, gate_up_concat: bool = False,
                      zero_tail: bool = False, status: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Gradient dH bf16 [rows, N] of ``silu_mul`` from dact bf16 [rows, N/2] and either H8 with
    H8_scale or H. ``act`` (bf16 [rows, N/2]) is computed again into the given buffer, and the
    weights' gradient into ``dweights`` (float32, indexed like the weights; 0 for a dropped
    assignment)."""
    if _native is not None:
        rc = _native.silu_mul_backward(dact, dH, H, H8, H8_scale, offs, row_of, weights, act,
                                       dweights, gate_up_concat, zero_tail, status, stream)
        if rc is not None:
            _raise(rc, "gg_silu_mul_backward")
            return dH
    _check(dact, "dact", _BF16, 2)
    rows, half = dact.shape
    N, dev = 2 * half, dact.get_device()
    if (H is None) == (H8 is None):
        raise ValueError("exactly one of H and H8 must be given")
    used, rp, n, wp, flags = _act_args(dact, offs, row_of, weights, gate_up_concat, zero_tail, dev)
    p8, ps = _args8(H8, H8_scale, rows, N, _half_blocks(N), dev)
    dH = _new(dH, (rows, N), _BF16, dact, stream)
    rc = lib().gg_silu_mul_backward(
        dact.data_ptr(), _arg(H, "H", (rows, N), _BF16, dev), p8, ps, rows, N, used, rp, n, wp,
        flags, _arg(dH, "dH", (rows, N), _BF16, dev),
        _arg(act, "act", (rows, half), _BF16, dev),
        _per_row(dweights, "dweights", rows if row_of is None else n, dev), _status_ptr(status),
        _stream_handle(stream, dev))
    _raise(rc, "gg_silu_mul_backward")
    return dH


def pack8(X: torch.Tensor, X8: Optional[torch.Tensor] = None,
          scale: Optional[torch.Tensor] = None, *, offs: Optional[torch.Tensor] = None,
          status: Optional[torch.Tensor] = None, stream=None):
    """The rows of X bf16 [rows, cols] in 8 bits: (X8 float8_e4m3fn [rows, cols], scale
    float8_e8m0fnu [rows, ceil(cols/32)]), X ~ X8 * scale with one power of two for 32 columns.
    Rows at and past the last of ``offs`` are not touched."""
    if _native is not None:
        rc = _native.pack8(X, X8, scale, offs, status, stream)
        if rc is not None:
            _raise(rc, "gg_pack8")
            return X8, scale
    _check(X, "X", _BF16, 2)
    rows, cols = X.shape
    codes, dev = (cols + BLOCK8 - 1) // BLOCK8, X.get_device()
    X8 = _new(X8, (rows, cols), _E4M3, X, stream)
    scale = _new(scale, (rows, codes), _E8M0, X, stream)
    rc = lib().gg_pack8(X.data_ptr(), rows, cols, _used_ptr(offs, False, dev),
                        _arg(X8, "X8", (rows, cols), _E4M3, dev),
                        _arg(scale, "scale", (rows, codes), _E8M0, dev), _status_ptr(status),
                        _stream_handle(stream, dev))
    _raise(rc, "gg_pack8")
    return X8, scale


def unpack8(X8: torch.Tensor, scale: torch.Tensor, X: Optional[torch.Tensor] = None, *,
            offs: Optional[torch.Tensor] = None, zero_tail: bool = False,
            status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """X bf16 [rows, cols] = X8 * scale, exact for what ``pack8`` wrote."""
    if _native is not None:
        rc = _native.unpack8(X8, scale, X, offs, zero_tail, status, stream)
        if rc is not None:
            _raise(rc, "gg_unpack8")
            return X
    _check(X8, "X8", _E4M3, 2)
    rows, cols = X8.shape
    dev = X8.get_device()
    X = _new(X, (rows, cols), _BF16, X8, stream)
    rc = lib().gg_unpack8(
        X8.data_ptr(), _arg(scale, "scale", (rows, (cols + BLOCK8 - 1) // BLOCK8), _E8M0, dev),
        rows, cols, _used_ptr(offs, zero_tail, dev), FLAG_ZERO_TAIL if zero_tail else 0,
        _arg(X, "X", (rows, cols), _BF16, dev), _status_ptr(status), _stream_handle(stream, dev))
    _raise(rc, "gg_unpack8")
    return X


# ---------------------------------------------------------------------------------- autograd

def _dense(g: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels take it: contiguous, on a 16-byte boundary."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, how, bias, num_tokens, status):
        ids, w = gate_topk(logits, k, bias=bias, num_tokens=num_tokens, status=status, **how)
        ctx.mark_non_differentiable(ids)
        ctx.save_for_backward(logits, ids)
        ctx.how, ctx.status = how, status
        return ids, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        logits, ids = ctx.saved_tensors
        dx = gate_topk_backward(logits, ids, dw.contiguous(), status=ctx.status, **ctx.how)
        return dx, None, None, None, None, None


def gate(logits: torch.Tensor, k: int, *, score: int = GATE_SOFTMAX, renorm: bool = True,
         scale: float = 1.0, bias: Optional[torch.Tensor] = None,
         num_tokens: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """``gate_topk`` with the gradient of the logits: (topk_ids, weights). The bias, which only
    takes part in the choice, has none."""
    how = {"score": score, "renorm": renorm, "scale": scale}
    if _wants_grad(logits):
        return _Gate.apply(logits, k, how, bias, num_tokens, status)
    return gate_topk(logits, k, bias=bias, num_tokens=num_tokens, status=status, **how)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, topk_ids, E, status):
        A, row_of, offs = route(topk_ids, X, E, status=status)
        ctx.mark_non_differentiable(row_of, offs)
        ctx.save_for_backward(row_of)
        ctx.k, ctx.status = topk_ids.shape[1], status
        return A, row_of, offs

    @staticmethod
    @once_differentiable
    def backward(ctx, dA, *_):
        return unroute(_dense(dA), ctx.saved_tensors[0], ctx.k, status=ctx.status), None, None, None


def dispatch(X: torch.Tensor, topk_ids: torch.Tensor, E: int, *,
             status: Optional[torch.Tensor] = None):
    """``route`` with the gradient of X (the sum over a token's packed rows): (A_packed, row_of,
    offs). Rows of A_packed past the last offset are uninitialised, as ``grouped_mm`` and
    ``expert_mlp`` expect."""
    if _wants_grad(X):
        return _Dispatch.apply(X, topk_ids, E, status)
    return route(topk_ids, X, E, status=status)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Y, row_of, k, weights, residual, offs, status):
        keep = Y if ctx.needs_input_grad[3] else None  # only the weights' gradient needs it
        ctx.save_for_backward(keep, row_of, weights, offs)
        ctx.k, ctx.rows, ctx.status = k, Y.shape[0], status
        return unroute(Y, row_of, k, weights=weights, residual=residual, status=status)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        Y, row_of, weights, offs = ctx.saved_tensors
        dY = dw = None
        if ctx.needs_input_grad[0]:
            make = torch.zeros if offs is None else torch.empty
            dY = make((ctx.rows, dout.shape[1]), dtype=_BF16, device=dout.device)
        if ctx.needs_input_grad[3]:
            dw = torch.empty_like(weights)
        if dY is not None or dw is not None:
            unroute_backward(_dense(dout), row_of, ctx.k, dY, Y=Y, weights=weights, dweights=dw,
                             offs=offs, zero_tail=offs is not None and dY is not None,
                             status=ctx.status)
        return dY, None, None, dw, dout if ctx.needs_input_grad[4] else None, None, None


def combine(Y: torch.Tensor, row_of: torch.Tensor, k: int, *,
            weights: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
            offs: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``unroute`` with the gradients of Y, the weights and the residual. With ``offs`` from
    ``route``, whose row_of names every row before the last offset, only the rows of dY past it
    are cleared; without, all of dY is. Y is kept for the backward pass only when the weights
    require a gradient; weights applied in ``swiglu`` or ``expert_mlp`` instead spare it."""
    if _wants_grad(Y, weights, residual):
        return _Combine.apply(Y, row_of, k, weights, residual, offs, status)
    return unroute(Y, row_of, k, weights=weights, residual=residual, status=status)


def _new8(H):
    rows, N = H.shape
    return (torch.empty((rows, N), dtype=_E4M3, device=H.device),
            torch.empty((rows, _half_blocks(N)), dtype=_E8M0, device=H.device))


class _SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, offs, row_of, weights, concat, ckpt8, status):
        H8, scale = _new8(H) if ckpt8 else (None, None)
        act = silu_mul(H, offs=offs, row_of=row_of, weights=weights, gate_up_concat=concat,
                       zero_tail=True, H8=H8, H8_scale=scale, status=status)
        ctx.save_for_backward(None if ckpt8 else H, H8, scale, offs, row_of, weights)
        ctx.concat, ctx.status = concat, status
        return act

    @staticmethod
    @once_differentiable
    def backward(ctx, dact):
        H, H8, scale, offs, row_of, weights = ctx.saved_tensors
        # without row_of the rows that are not in use have weights that no row depends on
        dw = torch.zeros_like(weights) if ctx.needs_input_grad[3] else None
        dH = silu_mul_backward(_dense(dact), H=H, H8=H8, H8_scale=scale, offs=offs,
                               row_of=row_of, weights=weights, dweights=dw,
                               gate_up_concat=ctx.concat, zero_tail=True, status=ctx.status)
        return dH, None, None, dw, None, None, None


def swiglu(H: torch.Tensor, offs: torch.Tensor, *, row_of: Optional[torch.Tensor] = None,
           weights: Optional[torch.Tensor] = None, gate_up_concat: bool = False,
           ckpt8: bool = False, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``silu_mul`` with the gradients of H and of the weights; rows past the last offset are
    zero in the result and in dH (a row_of names every row before it, as ``route``'s does; to
    drop an assignment, drop its id before ``route``). With ``ckpt8`` H is kept for the backward
    pass in 8 bits (e4m3, a power-of-two scale for 32 columns), and the gradients are those at
    these values."""
    if _wants_grad(H, weights):
        return _SwiGLU.apply(H, offs, row_of, weights, gate_up_concat, ckpt8, status)
    return silu_mul(H, offs=offs, row_of=row_of, weights=weights, gate_up_concat=gate_up_concat,
                    zero_tail=True, status=status)


def _products(A, W1, W2, offs, row_of, weights, concat, w_nk, ckpt8, status):
    """(H, H8, H8's scale, Y): A @ W1, with ckpt8 also in 8 bits, and the second product of its
    activation."""
    rows = A.shape[0]
    H = torch.empty((rows, W1.shape[1 if w_nk else 2]), dtype=_BF16, device=A.device)
    Y = torch.empty((rows, W2.shape[1 if w_nk else 2]), dtype=_BF16, device=A.device)
    forward_ex(A, W1, offs, H, w_nk=w_nk, status=status)
    H8, H8s = _new8(H) if ckpt8 else (None, None)
    act = silu_mul(H, offs=offs, row_of=row_of, weights=weights, gate_up_concat=concat, H8=H8,
                   H8_scale=H8s, status=status)
    forward_ex(act, W2, offs, Y, zero_tail=True, w_nk=w_nk, status=status)
    return H, H8, H8s, Y


class _ExpertMLP(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, W1, W2, offs, row_of, weights, concat, w_nk, ckpt8, status):
        H, H8, H8s, Y = _products(A, W1, W2, offs, row_of, weights, concat, w_nk,
                                  ckpt8, status)
        A8 = A8s = None
        keep = A if ctx.needs_input_grad[1] else None  # A is only needed for W1's gradient
        if ckpt8 and keep is not None:
            A8, A8s = pack8(A, offs=offs, status=status)
            keep = None
        ctx.save_for_backward(keep, A8, A8s, None if ckpt8 else H, H8, H8s, W1, W2, offs, row_of,
                              weights)
        ctx.concat, ctx.w_nk, ctx.status = concat, w_nk, status
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        A, A8, A8s, H, H8, H8s, W1, W2, offs, row_of, weights = ctx.saved_tensors
        need, st, w_nk = ctx.needs_input_grad, ctx.status, ctx.w_nk
        dY = _dense(dY)
        rows, half = dY.shape[0], W2.shape[2 if w_nk else 1]
        dA = dW1 = dW2 = dw = act = None
        dact = torch.empty((rows, half), dtype=_BF16, device=dY.device)
        dgrad_ex(dY, W2, offs, dact, w_nk=w_nk, status=st)
        if need[2]:
            act = torch.empty_like(dact)
        if need[5]:
            dw = torch.zeros_like(weights)
        dH = silu_mul_backward(dact, H=H, H8=H8, H8_scale=H8s, offs=offs, row_of=row_of,
                               weights=weights, act=act, dweights=dw, gate_up_concat=ctx.concat,
                               status=st)
        if need[2]:
            dW2 = torch.empty_like(W2)
            wgrad_ex(act, dY, offs, dW2, w_nk=w_nk, status=st)
        if need[1]:
            if A8 is not None:
                A = unpack8(A8, A8s, offs=offs, status=st)
            dW1 = torch.empty_like(W1)
            wgrad_ex(A, dH, offs, dW1, w_nk=w_nk, status=st)
        if need[0]:
            dA = torch.empty((rows, W1.shape[2 if w_nk else 1]), dtype=_BF16, device=dY.device)
            dgrad_ex(dH, W1, offs, dA, zero_tail=True, w_nk=w_nk, status=st)
        return dA, dW1, dW2, None, None, dw, None, None, None, None


def expert_mlp(A: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, offs: torch.Tensor, *,
               row_of: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
               gate_up_concat: bool = False, w_nk: bool = False, ckpt8: bool = False,
               status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = (weight * silu(gate) * up) @ W2[e] with gate and up the columns of A @ W1[e]: both
    expert products and the activation between them, with the gradients of A, W1, W2 and the
    weights. A bf16 [rows, K], W1 bf16 [E, K, N], W2 bf16 [E, N/2, K2] (``w_nk``: [E, N, K] and
    [E, K2, N/2]); row_of and weights as in ``swiglu`` (the weights applied before the second
    product: their gradient then needs no copy of Y). Rows past the last offset are zero in Y
    and dA.

    The backward pass computes the activation again, so only A and A @ W1 are kept for it; with
    ``ckpt8`` both in 8 bits (half their bytes), and the gradients are those at these values."""
    if _wants_grad(A, W1, W2, weights):
        return _ExpertMLP.apply(A, W1, W2, offs, row_of, weights, gate_up_concat, w_nk, ckpt8,
                                status)
    return _products(A, W1, W2, offs, row_of, weights, gate_up_concat, w_nk, False, status)[3]
