"""float64 definitions (numpy) of the operators in front of a conditional circuit: layer norm, linear attention with
a decay for each head, the orthogonalised update, the heads' norm with rotation, softmax attention -- and their
gradients.  Test infrastructure only."""
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


def rotary(x, positions, freq, interleaved=False, magnitude=1.0, norm=False, w=None, eps=1e-6, way=1.0):
    """x [T, H, d]: root mean square norm of every head, then its first 2 len(freq) elements turned as pairs."""
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    n = len(freq)
    a, b = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    angle = np.asarray(positions, np.float64)[:, None, None] * freq
    c, s = magnitude * np.cos(angle), way * magnitude * np.sin(angle)
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def rotary_grad(dy, x, positions, freq, interleaved=False, magnitude=1.0, norm=False, w=None, eps=1e-6):
    """(dx, dw)"""
    h = rotary(dy, positions, freq, interleaved, magnitude, way=-1.0)
    if not norm:
        return h, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dw = (h * n).sum((0, 1))
    g = h * (1.0 if w is None else w)
    return r * (g - n * (g * n).mean(-1, keepdims=True)), dw


def _scores(q, k, scale, past):
    """[H, n, m] scores of n queries behind `past` of the m keys; -inf where a key lies behind its query."""
    k = np.repeat(k, q.shape[1] // k.shape[1], 1)
    x = np.einsum("ihd,jhd->hij", q, k) * scale
    x[:, np.arange(len(k))[None] > past + np.arange(len(q))[:, None]] = -np.inf
    return x


def attend(q, k, v, scale, past=0):
    """(o, lse) of one sequence: q [n, H, dk] behind `past` of the keys k, v [past + n, K, .]."""
    x = _scores(q, k, scale, past)
    top = x.max(-1, keepdims=True)
    p = np.exp(x - top)
    total = p.sum(-1, keepdims=True)
    o = np.einsum("hij,jhd->ihd", p / total, np.repeat(v, q.shape[1] // v.shape[1], 1))
    return o, (top + np.log(total))[..., 0].T


def softmax_attention(q, k, v, cu, scale):
    """Causal attention along every sequence; tokens outside all of them: 0."""
    T, H, _ = q.shape
    o, lse = np.zeros((T, H, v.shape[2])), np.zeros((T, H))
    for a, b in zip(cu[:-1], cu[1:]):
        if b > a:
            o[a:b], lse[a:b] = attend(q[a:b], k[a:b], v[a:b], scale)
    return o, lse


def softmax_attention_grad(do, q, k, v, o, lse, cu, scale):
    """(dq, dk, dv) of the o and lse that are given."""
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    H, K = q.shape[1], k.shape[1]
    for a, b in zip(cu[:-1], cu[1:]):
        if b == a:
            continue
        qq, g = q[a:b], do[a:b]
        kk, vv = (np.repeat(t[a:b], H // K, 1) for t in (k, v))
        p = np.exp(_scores(qq, k[a:b], scale, 0) - lse[a:b].T[..., None])
        ds = p * (np.einsum("ihd,jhd->hij", g, vv) - (g * o[a:b]).sum(-1).T[..., None])
        dq[a:b] = scale * np.einsum("hij,jhd->ihd", ds, kk)
        dkk, dvv = scale * np.einsum("hij,ihd->jhd", ds, qq), np.einsum("hij,ihd->jhd", p, g)
        dk[a:b], dv[a:b] = (t.reshape(b - a, K, H // K, -1).sum(2) for t in (dkk, dvv))
    return dq, dk, dv
