"""fp64 definitions of the operators around the grouped GEMM (numpy, plain and slow).

Inputs are float64 arrays (bf16 or fp32 values widened exactly) and int arrays; results are
float64. Test infrastructure, like the rest of this package.

  gate      k experts of each token and their weights from its logits, and the gradient
  unroute   out[t] = residual[t] + sum_s w[t, s] Y[row_of[t k + s]], and the gradients
  pack8     rows in e4m3 with a power-of-two scale for 32 columns: the values they stand for
  silu_mul  weight * silu(gate) * up, and the gradients
"""
from __future__ import annotations

import numpy as np


def _softmax(x):
    """Over the last axis; -inf carries nothing, a row of only -inf is 0."""
    m = x.max(-1, keepdims=True)
    e = np.exp(x - np.where(np.isneginf(m), 0, m))
    s = e.sum(-1, keepdims=True)
    return e / np.where(s > 0, s, 1)


def _log_sigmoid(x):
    return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))


def _mask(x):
    """NaN and +inf count as masked."""
    return np.where(x < np.inf, x, -np.inf)


def gate(x, k, sigmoid=False, renorm=True, scale=1.0, bias=None, num_tokens=None):
    """(ids [T, k], weights [T, k]) of logits x [T, E]."""
    x = _mask(np.asarray(x, np.float64)).copy()
    T, E = x.shape
    if num_tokens is not None:
        x[max(0, min(T, num_tokens)):] = -np.inf
    key = x
    if bias is not None:
        b = _mask(np.asarray(bias, np.float64))
        key = np.where(np.isneginf(x) | np.isneginf(b), -np.inf, np.exp(_log_sigmoid(x)) + b)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]  # equal keys: the lowest expert first
    ids = np.where(np.take_along_axis(key, ids, 1) > -np.inf, ids, -1)
    return ids, scale * _weights(x, ids, sigmoid, renorm)


def _weights(x, ids, sigmoid, renorm):
    xs = np.where(ids >= 0, np.take_along_axis(x, np.maximum(ids, 0), 1), -np.inf)
    if renorm:
        return _softmax(_log_sigmoid(xs) if sigmoid else xs)
    if sigmoid:
        return np.exp(_log_sigmoid(xs))
    m = x.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0, m)
    s = np.exp(x - m).sum(1, keepdims=True)
    return np.exp(xs - m) / np.where(s > 0, s, 1)


def gate_backward(x, ids, dw, sigmoid=False, renorm=True, scale=1.0):
    """Gradient of the logits: the Jacobian of the weights, slot by slot."""
    x = _mask(np.asarray(x, np.float64))
    T, E = x.shape
    v = _weights(x, ids, sigmoid, renorm)
    dx = np.zeros((T, E))
    p = _softmax(x)
    for t in range(T):
        live = [s for s in range(ids.shape[1]) if ids[t, s] >= 0 and x[t, ids[t, s]] > -np.inf]
        for s in live:  # the derivative of weight s with respect to every logit
            g = scale * dw[t, s]
            if sigmoid:
                inner = lambda r: np.exp(_log_sigmoid(-x[t, ids[t, r]]))  # noqa: E731
                dx[t, ids[t, s]] += g * v[t, s] * inner(s)
                if renorm:
                    for r in live:
                        dx[t, ids[t, r]] -= g * v[t, s] * v[t, r] * inner(r)
            else:
                dx[t, ids[t, s]] += g * v[t, s]
                if renorm:
                    for r in live:
                        dx[t, ids[t, r]] -= g * v[t, s] * v[t, r]
                else:
                    dx[t] -= g * v[t, s] * p[t]
    return dx


def unroute(Y, row_of, k, weights=None, residual=None):
    T = len(row_of) // k
    out = np.zeros((T, Y.shape[1])) if residual is None else np.array(residual, np.float64)
    for i, r in enumerate(row_of):
        if 0 <= r < len(Y):
            out[i // k] += Y[r] * (1.0 if weights is None else weights.reshape(-1)[i])
    return out


def unroute_backward(dout, Y, row_of, k, weights=None):
    """(dY with zeros where no entry points, dweights [T, k])."""
    dY, dw = np.zeros(Y.shape), np.zeros(len(row_of))
    for i, r in enumerate(row_of):
        if 0 <= r < len(Y):
            dY[r] = dout[i // k] * (1.0 if weights is None else weights.reshape(-1)[i])
            dw[i] = dout[i // k] @ Y[r]
    return dY, dw.reshape(-1, k)


E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(8)][:127])  # without the NaN code


def round_e4m3(v):
    """Nearest e4m3 value, ties to the even code, |v| <= 448."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 0, len(E4M3) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(E4M3[pick], v)


def pack8(x):
    """(values, codes): the 8-bit form of the rows x [R, C], block by block of 32 columns."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    out, codes = np.empty((R, C)), np.zeros((R, -(-C // 32)), np.int64)
    for j in range(codes.shape[1]):
        b = x[:, 32 * j:32 * j + 32]
        top = np.where(np.isfinite(b), np.abs(b), 0).max(1)
        code = np.full(R, 9)
        for c in range(9, 247):  # the least code that brings the block into range
            code = np.where(top > 448.0 * 2.0 ** (c - 127), c + 1, code)
        s = 2.0 ** (code - 127)[:, None]
        top = np.where(code == 247, 240.0, 448.0)[:, None]  # 256 * 2^120 is past bf16's range
        with np.errstate(invalid="ignore"):
            out[:, 32 * j:32 * j + 32] = np.where(
                np.isfinite(b),
                round_e4m3(np.clip(np.where(np.isfinite(b), b, 0) / s, -top, top)) * s, np.nan)
        codes[:, j] = code
    return out, codes


def halves(N, concat):
    """Column numbers of gate and up."""
    j = np.arange(N // 2)
    if concat:
        return j, j + N // 2
    return j // 128 * 256 + j % 128, j // 128 * 256 + j % 128 + 128


def pack8_halves(H, concat):
    """The 8-bit values of H with gate and up columns in blocks of their own."""
    g, u = halves(H.shape[1], concat)
    out = np.empty(H.shape)
    out[:, g], out[:, u] = pack8(H[:, g])[0], pack8(H[:, u])[0]
    return out


def silu_mul(H, concat, w=None):
    g, u = (H[:, c] for c in halves(H.shape[1], concat))
    with np.errstate(over="ignore"):
        a = g / (1 + np.exp(-g)) * u
    return a if w is None else a * w[:, None]


def silu_mul_backward(dact, H, concat, w=None):
    """(dH, dweights [rows])."""
    cg, cu = halves(H.shape[1], concat)
    g, u = H[:, cg], H[:, cu]
    with np.errstate(over="ignore"):
        q = 1 / (1 + np.exp(-g))
    d = dact if w is None else dact * w[:, None]
    dH = np.empty(H.shape)
    dH[:, cg] = d * u * (q + g * q * (1 - q))
    dH[:, cu] = d * g * q
    return dH, (dact * g * q * u).sum(1)
