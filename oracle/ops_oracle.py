"""float64 definitions (numpy) of the operators in front of a conditional circuit: layer norm, linear attention with
a decay for each head, the orthogonalised update -- and their gradients.  Test infrastructure only."""
from __future__ import annotations

import numpy as np


def layer_norm(x, w=None, b=None, eps=1e-5):
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    y = (x - mean) * rstd * (1.0 if w is None else w) + (0.0 if b is None else b)
    return y, mean[:, 0], rstd[:, 0]


def layer_norm_grad(dy, x, mean, rstd, w=None):
    n = (x - mean[:, None]) * rstd[:, None]
    g = dy * (1.0 if w is None else w)
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


def _decay(log_decay):
    return np.exp(log_decay)[:, None, None]


def linear_attention(q, k, v, log_decay, cu, scale, state=None):
    """Token by token; q [T, H, dk], k, v [T, K, .], state [n, H, dk, dv].  Tokens outside every sequence: 0."""
    T, H, dk = q.shape
    grp, dv = H // k.shape[1], v.shape[2]
    kk, vv, lam = np.repeat(k, grp, 1), np.repeat(v, grp, 1), _decay(log_decay)
    o = np.zeros((T, H, dv))
    out = np.zeros((len(cu) - 1, H, dk, dv)) if state is None else state.copy()
    for s in range(len(cu) - 1):
        S = out[s]
        for t in range(cu[s], cu[s + 1]):
            S = lam * S + kk[t][:, :, None] * vv[t][:, None, :]
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
        out[s] = S
    return o, out


def linear_attention_grad(do, q, k, v, log_decay, cu, scale, state=None, dstate=None):
    T, H, dk = q.shape
    K, dv = k.shape[1], v.shape[2]
    grp = H // K
    kk, vv, lam = np.repeat(k, grp, 1), np.repeat(v, grp, 1), _decay(log_decay)
    dq, dkk, dvv = np.zeros((T, H, dk)), np.zeros((T, H, dk)), np.zeros((T, H, dv))
    n = len(cu) - 1
    out = np.zeros((n, H, dk, dv)) if dstate is None else dstate.copy()
    for s in range(n):
        S = np.zeros((H, dk, dv)) if state is None else state[s].copy()
        for t in range(cu[s], cu[s + 1]):
            S = lam * S + kk[t][:, :, None] * vv[t][:, None, :]
            dq[t] = scale * np.einsum("hkv,hv->hk", S, do[t])
        D = out[s]
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            now = D + scale * q[t][:, :, None] * do[t][:, None, :]
            dkk[t] = np.einsum("hkv,hv->hk", now, vv[t])
            dvv[t] = np.einsum("hk,hkv->hv", kk[t], now)
            D = lam * now
        out[s] = D
    return dq, dkk.reshape(T, K, grp, dk).sum(2), dvv.reshape(T, K, grp, dv).sum(2), out


def orthogonalize(g, coefficients, eps, operands=lambda step: (lambda x: x,) * 3):
    """Newton-Schulz steps on one matrix; operands(step): the rounding of the operands of A = X X^T, A A and B X."""
    tall = g.shape[0] > g.shape[1]
    x = g.T if tall else g
    x = x / (np.sqrt((x * x).sum()) + eps)
    for step, (a, b, c) in enumerate(coefficients):
        gram, square, apply = operands(step)
        A = gram(x) @ gram(x).T
        x = a * x + apply(b * A + c * (square(A) @ square(A))) @ apply(x)
    return x.T if tall else x
