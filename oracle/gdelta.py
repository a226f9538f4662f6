"""Plain CPU oracle for the gated delta rule and for layer norm.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it imports nothing
from the product.  Everything is float64.  The gated delta rule is evaluated
token by token (nothing is chunked), and its backward is the step-by-step
reverse-time adjoint; with k^, q^ the unit-length key and query, head h
reading group h // (heads / groups), alpha = exp(g):

  u_t = beta_t (v_t - alpha_t S_{t-1} k^_t),  S_t = alpha_t S_{t-1} + u_t k^_t^T,  y_t = scale S_t q^_t
  g_t = -exp(a_log) softplus(a_raw_t + dt_bias),  beta_t = sigmoid(b_raw_t)
"""
from __future__ import annotations

import numpy as np


def _gates(a_raw, b_raw, a_log, dt_bias):
    z = a_raw + dt_bias
    sp = np.logaddexp(0.0, z)
    rate = np.exp(a_log)
    return z, sp, rate, np.exp(-rate * sp), 1.0 / (1.0 + np.exp(-b_raw))


def _unit(x, eps):
    r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) + eps)
    return x * r, r


def _f64(*xs):
    return [None if x is None else np.asarray(x, np.float64) for x in xs]


def forward(q, k, v, a_raw, b_raw, a_log, dt_bias, h0=None, scale=0.0, eps=1e-6):
    """y [B, T, H, V] and the last state [B, H, V, K]."""
    q, k, v, a_raw, b_raw, a_log, dt_bias, h0 = _f64(q, k, v, a_raw, b_raw, a_log, dt_bias, h0)
    B, T, H, V = v.shape
    K, share = k.shape[3], H // k.shape[2]
    scale = scale or K ** -0.5
    qn, kn = (np.repeat(_unit(x, eps)[0], share, 2) for x in (q, k))
    _, _, _, alpha, beta = _gates(a_raw, b_raw, a_log, dt_bias)
    S = np.zeros((B, H, V, K)) if h0 is None else h0.copy()
    y = np.empty_like(v)
    for t in range(T):
        S = alpha[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhvk,bhk->bhv", S, kn[:, t]))
        S = S + u[..., None] * kn[:, t, :, None, :]
        y[:, t] = scale * np.einsum("bhvk,bhk->bhv", S, qn[:, t])
    return y, S


def backward(dy, q, k, v, a_raw, b_raw, a_log, dt_bias, h0=None, scale=0.0, eps=1e-6):
    """Gradients of sum(dy * y) for every input but h0, as a dict."""
    dy, q, k, v, a_raw, b_raw, a_log, dt_bias, h0 = _f64(dy, q, k, v, a_raw, b_raw, a_log, dt_bias, h0)
    B, T, H, V = v.shape
    G, K = k.shape[2], k.shape[3]
    share = H // G
    scale = scale or K ** -0.5
    (q1, rq), (k1, rk) = _unit(q, eps), _unit(k, eps)
    qn, kn = np.repeat(q1, share, 2), np.repeat(k1, share, 2)
    z, sp, rate, alpha, beta = _gates(a_raw, b_raw, a_log, dt_bias)
    states, miss = [np.zeros((B, H, V, K)) if h0 is None else h0], []
    for t in range(T):
        aS = alpha[:, t, :, None, None] * states[-1]
        miss.append(v[:, t] - np.einsum("bhvk,bhk->bhv", aS, kn[:, t]))
        states.append(aS + (beta[:, t, :, None] * miss[-1])[..., None] * kn[:, t, :, None, :])
    dqn, dkn, dv = np.empty_like(qn), np.empty_like(kn), np.empty_like(v)
    dalpha, dbeta = np.empty_like(alpha), np.empty_like(beta)
    dS = np.zeros((B, H, V, K))
    for t in reversed(range(T)):
        d, kt, a = scale * dy[:, t], kn[:, t], alpha[:, t, :, None, None]
        dqn[:, t] = np.einsum("bhv,bhvk->bhk", d, states[t + 1])
        dS = dS + d[..., None] * qn[:, t, :, None, :]
        du = np.einsum("bhvk,bhk->bhv", dS, kt)
        dbeta[:, t] = (du * miss[t]).sum(-1)
        dv[:, t] = beta[:, t, :, None] * du
        u = beta[:, t, :, None] * miss[t]
        dkn[:, t] = np.einsum("bhvk,bhv->bhk", dS, u) - np.einsum("bhvk,bhv->bhk", a * states[t], dv[:, t])
        dS = dS - dv[:, t][..., None] * kt[:, :, None, :]      # now the gradient of alpha S_{t-1}
        dalpha[:, t] = (dS * states[t]).sum((-1, -2))
        dS = a * dS

    def raw(d, n, r):
        d = d.reshape(B, T, G, share, K).sum(3)
        return r * (d - n * (d * n).sum(-1, keepdims=True))

    dg = dalpha * alpha
    dz = -rate * dg / (1.0 + np.exp(-z))
    return dict(q=raw(dqn, q1, rq), k=raw(dkn, k1, rk), v=dv, a_raw=dz, b_raw=dbeta * beta * (1.0 - beta),
                a_log=(-rate * sp * dg).sum((0, 1)), dt_bias=dz.sum((0, 1)))


def layernorm_forward(x, w=None, b=None, eps=1e-5):
    """y, mean, rstd."""
    x, w, b = _f64(x, w, b)
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    y = y if w is None else y * w
    return (y if b is None else y + b), mean, rstd


def layernorm_backward(dy, x, w=None, d_add=None, mean=None, rstd=None, eps=1e-5):
    """dx, dw, db (mean and rstd: those the backward is given, else the row's own)."""
    dy, x, w, d_add, mean, rstd = _f64(dy, x, w, d_add, mean, rstd)
    if mean is None:
        _, mean, rstd = layernorm_forward(x, eps=eps)
    n = (x - mean[:, None]) * rstd[:, None]
    dn = dy if w is None else dy * w
    dx = rstd[:, None] * (dn - dn.mean(1, keepdims=True) - n * (dn * n).mean(1, keepdims=True))
    return (dx if d_add is None else dx + d_add), (dy * n).sum(0), dy.sum(0)
