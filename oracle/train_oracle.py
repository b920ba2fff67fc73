"""Plain numpy float64 gradients of the layer's steps, and the AdamW step.

Written from the forward formulas of ``moe_oracle`` by the rules of calculus,
one function per step:

  out[t] = sum_j w[t,j] y[pos[t,j]]          combine_backward
  y = W2 act(W1 x + b1) + b2                 expert_ffn_backward
  x_perm[pos[s]] = x[s // K]                 dispatch_backward

``adamw`` is the decoupled-decay Adam step of Loshchilov and Hutter (Decoupled
Weight Decay Regularization, algorithm 2) with the schedule factor 1 and the
decay scaled by the learning rate.  ``encode_e4m3`` rounds to the 8-bit floating-point
format with 4 exponent and 3 mantissa bits (bias 7, largest value 448).
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erf as _erf


def gelu_slope(a):
    """GELU'(a) = Phi(a) + a phi(a)."""
    return 0.5 * (1.0 + _erf(a / math.sqrt(2.0))) + a * np.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)


def sigmoid(a):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-a))


def silu_slope(a):
    """SiLU'(a) = s + a s (1 - s), s = sigmoid(a)."""
    s = sigmoid(a)
    return s + a * s * (1.0 - s)


def combine_backward(dout, y_perm, pos, w):
    """(dy_perm [R, H], dw [T, K]) for the R rows of ``y_perm``; a dropped
    slot's dw is 0, a row no slot holds stays 0."""
    T, K = w.shape
    dy = np.zeros(y_perm.shape)
    dw = np.zeros((T, K))
    p = np.asarray(pos).reshape(T, K)
    for t in range(T):
        for j in range(K):
            if p[t, j] >= 0:
                dy[p[t, j]] = w[t, j] * dout[t]
                dw[t, j] = dout[t] @ y_perm[p[t, j]]
    return dy, dw


def dispatch_backward(dx_perm, pos, T, K, add=None):
    dx = np.zeros((T, dx_perm.shape[1])) if add is None else np.array(add, dtype=np.float64)
    p = np.asarray(pos).reshape(T, K)
    for j in range(K):
        kept = p[:, j] >= 0
        dx[kept] += dx_perm[p[kept, j]]
    return dx


def expert_ffn_backward(x, h, dy, W1, W2, b1=None, act="gelu"):
    """One expert's gradients from its rows ``x [n, H]``, the kept ``h [n, F]``
    and ``dy [n, H]``: dict with a, dh, da, dx, dW1, db1, dW2, db2."""
    a = x @ W1.T + (0.0 if b1 is None else b1)
    dh = dy @ W2
    if act == "swiglu":
        F = W2.shape[1]
        g, u = a[:, :F], a[:, F:]
        da = np.concatenate([dh * u * silu_slope(g), dh * g * sigmoid(g)], axis=1)
    else:
        da = dh * gelu_slope(a)
    return dict(a=a, dh=dh, da=da, dx=da @ W1, dW1=da.T @ x, db1=da.sum(0), dW2=dy.T @ h, db2=dy.sum(0))


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, weight_decay):
    """(p, m, v) after one step."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p - lr * weight_decay * p - lr * hat, m, v


def e4m3_values():
    """The 127 non-negative finite values, in code order 0 .. 126."""
    return np.array([(c & 7) / 8.0 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3) - 7)
                     for c in range(127)])


def encode_e4m3(x):
    """Codes of x (|x| rounded to nearest, ties to the even code, at most 448)."""
    val = e4m3_values()
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(val, mag), 1, 126)
    lo = hi - 1
    below, above = mag - val[lo], val[hi] - mag
    code = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def decode_e4m3(code):
    c = np.asarray(code)
    return np.where(c & 128, -1.0, 1.0) * e4m3_values()[c & 127]
