"""float64 reference of the block's parts that serving and per-head norms need: the short
convolution with a carried history, and group norm with a SiLU gate, each with its backward.

TEST INFRASTRUCTURE ONLY -- see the package docstring.  Plain numpy from the definitions;
the convolution's own definition (tap i weights the input 3 - i steps back) is
m2rnn_block's, run over the history and the inputs in one.

Layouts: x, dout [B, T, C]; hist [B, 3, C], oldest first; w [C, 4]; bias [C];
y, g_pre [rows, D]; gamma, beta [D].
"""
from __future__ import annotations

import numpy as np

from .m2rnn_block import conv_silu, conv_silu_backward, silu, silu_grad

_f64 = np.float64


def conv_carry(x, w, bias=None, hist=None, lens=None):
    """(out [B, T, C], the last three inputs of each sequence's first lens[b] ones, history
    included [B, 3, C])."""
    x = np.asarray(x, _f64)
    B, T, C = x.shape
    h = np.zeros((B, 3, C), _f64) if hist is None else np.asarray(hist, _f64)
    full = np.concatenate([h, x], axis=1)
    out = conv_silu(full, w, bias)[:, 3:]
    lens = [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]
    return out, np.stack([full[b, n:n + 3] for b, n in enumerate(lens)])


def conv_carry_backward(x, w, bias, hist, dout):
    """Gradients of sum(dout out): (dx, dw, dbias or None, dhist)."""
    x, dout = np.asarray(x, _f64), np.asarray(dout, _f64)
    B, T, C = x.shape
    h = np.zeros((B, 3, C), _f64) if hist is None else np.asarray(hist, _f64)
    d = np.concatenate([np.zeros((B, 3, C), _f64), dout], axis=1)
    dfull, dw, db = conv_silu_backward(np.concatenate([h, x], axis=1), w, bias, d)
    return dfull[:, 3:], dw, db, dfull[:, :3]


def _normalise(y, groups, eps):
    y = np.asarray(y, _f64)
    g = y.reshape(y.shape[0], groups, -1)
    rs = 1.0 / np.sqrt(np.var(g, axis=-1, keepdims=True) + eps)
    return (g - np.mean(g, axis=-1, keepdims=True)) * rs, rs


def groupnorm_gate(y, g_pre, gamma, beta, groups, eps):
    """(gamma z + beta) SiLU(g_pre), z normalised over each group of channels."""
    z, _ = _normalise(y, groups, eps)
    return (np.asarray(gamma, _f64) * z.reshape(np.shape(y)) + beta) * silu(g_pre)


def groupnorm_gate_backward(y, g_pre, gamma, beta, groups, eps, dout):
    """Gradients of sum(dout out): (dy, dg_pre, dgamma, dbeta)."""
    z, rs = _normalise(y, groups, eps)
    zf = z.reshape(np.shape(y))
    gamma, dout = np.asarray(gamma, _f64), np.asarray(dout, _f64)
    da = dout * silu(g_pre)
    dz = (da * gamma).reshape(z.shape)
    dy = rs * (dz - dz.mean(-1, keepdims=True) - z * (dz * z).mean(-1, keepdims=True))
    return (dy.reshape(np.shape(y)), dout * (gamma * zf + beta) * silu_grad(g_pre),
            np.sum(da * zf, axis=0), np.sum(da, axis=0))
