"""float64 reference of the selective state-space scan: the linear sibling of the
M²RNN recurrence in the same layout.

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Plain numpy, token by token
from the definition, no blocking or reordering:

    d_t = softplus(logit_t + beta_n),  f_t = exp(-alpha_n d_t),
    H_t = f_t H_{t-1} + d_t k_t v_t^T,  y_t = H_t^T q_t + w_r[n] (.) v_t

and its chain rule walked from the last token to the first.  logit = -inf gives d = 0 and
f = 1: such a token leaves the state alone.

Layouts: k, q [B, T, NQ, K] (value head n reads head n // (N // NQ)); v, dy
[B, T, N, V]; logit [B, T, N]; alpha, beta [N]; w_r [N, V]; H0, dHT [B, N, K, V].
"""
from __future__ import annotations

import numpy as np

_f64 = np.float64


def _a(x):
    return None if x is None else np.asarray(x, dtype=_f64)


def _softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def _sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def ssm_forward(k, v, q, logit, alpha, beta, w_r, H0=None):
    """(y [B, T, N, V], H_T [B, N, K, V], every state [T + 1, B, N, K, V])."""
    k, v, q, logit, alpha, beta, w_r, H0 = map(_a, (k, v, q, logit, alpha, beta, w_r, H0))
    B, T, NQ, K = k.shape
    N, V = v.shape[2:]
    G = N // NQ if NQ else 1
    d = _softplus(logit + beta)
    f = np.exp(-alpha * d)
    H = np.zeros((B, N, K, V), _f64) if H0 is None else H0.copy()
    y = np.empty((B, T, N, V), _f64)
    states = np.empty((T + 1, B, N, K, V), _f64)
    states[0] = H
    for t in range(T):
        kt, qt = np.repeat(k[:, t], G, axis=1), np.repeat(q[:, t], G, axis=1)
        H = (f[:, t, :, None, None] * H
             + d[:, t, :, None, None] * kt[:, :, :, None] * v[:, t, :, None, :])
        y[:, t] = np.einsum("bnkv,bnk->bnv", H, qt) + w_r * v[:, t]
        states[t + 1] = H
    return y, H, states


def ssm_backward(k, v, q, logit, alpha, beta, w_r, H0, dy, dHT=None):
    """Gradients of sum(dy y) + sum(dHT H_T): a dict with dk, dv, dq, dlogit, dw_r, dalpha,
    dbeta, dH0."""
    _, _, states = ssm_forward(k, v, q, logit, alpha, beta, w_r, H0)
    k, v, q, logit, alpha, beta, w_r, dy, dHT = map(
        _a, (k, v, q, logit, alpha, beta, w_r, dy, dHT))
    B, T, NQ, K = k.shape
    N, V = v.shape[2:]
    G = N // NQ if NQ else 1
    x = logit + beta
    d = _softplus(x)
    f = np.exp(-alpha * d)
    R = np.zeros((B, N, K, V), _f64) if dHT is None else dHT.copy()
    dk, dq = np.zeros((B, T, NQ, K), _f64), np.zeros((B, T, NQ, K), _f64)
    dv = np.empty_like(v)
    dd, dl = np.empty_like(x), np.empty_like(x)
    for t in range(T - 1, -1, -1):
        kt, qt = np.repeat(k[:, t], G, axis=1), np.repeat(q[:, t], G, axis=1)
        R = R + qt[:, :, :, None] * dy[:, t, :, None, :]
        dqh = np.einsum("bnkv,bnv->bnk", states[t + 1], dy[:, t])
        rv = np.einsum("bnkv,bnv->bnk", R, v[:, t])
        dkh = d[:, t, :, None] * rv
        dq[:, t] = dqh.reshape(B, NQ, G, K).sum(2)
        dk[:, t] = dkh.reshape(B, NQ, G, K).sum(2)
        dv[:, t] = d[:, t, :, None] * np.einsum("bnkv,bnk->bnv", R, kt) + w_r * dy[:, t]
        dd[:, t] = np.einsum("bnk,bnk->bn", rv, kt)
        dl[:, t] = f[:, t] * np.einsum("bnkv,bnkv->bn", R, states[t])
        R = f[:, t, :, None, None] * R
    dx = _sigmoid(x) * (dd - alpha * dl)
    return {"dk": dk, "dv": dv, "dq": dq, "dlogit": dx, "dw_r": np.einsum("btnv,btnv->nv", dy, v),
            "dalpha": np.sum(-d * dl, axis=(0, 1)), "dbeta": np.sum(dx, axis=(0, 1)), "dH0": R}


def ssm_step(H, k, v, q, logit, alpha, beta, w_r):
    """One token of every sequence: (y [B, N, V], the new state)."""
    y, HT, _ = ssm_forward(np.asarray(k)[:, None], np.asarray(v)[:, None], np.asarray(q)[:, None],
                           np.asarray(logit)[:, None], alpha, beta, w_r, H)
    return y[:, 0], HT
