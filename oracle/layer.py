"""fp64 definitions of the layer's operators around the channel-wise mixer: the gated delta
rule with scalar gates (snilld.dk, "Hvad Gated DeltaNet-2 aendrer": what the channel-wise rule
falls back to), layer norm over the residual sum, and the gradients of the norm and of the
short convolution.  Plain loops and sums over numpy arrays; no code is shared with the GPU
path."""
from __future__ import annotations

import numpy as np


def gdr_forward(q, k, v, g, beta, S0=None, scale=1.0):
    """One sequence, token by token: q, k [T, H_k, d_k], v [T, H_v, d_v], g, beta [T, H_v]; returns
    (o [T, H_v, d_v], S_T [H_v, d_k, d_v])."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    S = np.zeros((Hv, dk, dv)) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.zeros((T, Hv, dv))
    head = np.arange(Hv) // (Hv // Hk) if Hv else np.arange(0)
    for t in range(T):
        kt, qt = k[t, head], q[t, head]
        S = np.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - np.einsum("hk,hkv->hv", kt, S))
        S = S + kt[:, :, None] * u[:, None, :]
        o[t] = scale * np.einsum("hk,hkv->hv", qt, S)
    return o, S


def layer_norm(s, weight, bias=None, eps=1e-5):
    """(y, mean, rstd) of the rows of s [rows, cols]."""
    mean = s.mean(-1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(-1) + eps)
    y = (s - mean[:, None]) * rstd[:, None] * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(dy, s, weight, mean, rstd, ds=None):
    """(dx, dweight, dbias) with the statistics given."""
    xh = (s - mean[:, None]) * rstd[:, None]
    h = dy * weight
    dx = rstd[:, None] * (h - h.mean(-1, keepdims=True) - xh * (h * xh).mean(-1, keepdims=True))
    return (dx if ds is None else dx + ds), (dy * xh).sum(0), dy.sum(0)


def short_conv_backward(dy, x, weight, hist=None, dhist_out=None):
    """Gradients for one sequence: dy, x [T, C], weight [C, 4], hist, dhist_out [3, C] or None; returns
    (dx, dweight, dbias, dhist)."""
    T, C = x.shape
    ext = np.concatenate([np.zeros((3, C)) if hist is None else hist, x])  # [history | tokens]
    dext = np.zeros_like(ext)
    dw = np.zeros((C, 4))
    for t in range(T):
        for j in range(4):
            dext[t + j] += weight[:, j] * dy[t]
            dw[:, j] += dy[t] * ext[t + j]
    if dhist_out is not None:
        dext[T:T + 3] += dhist_out
    return dext[3:], dw, dy.sum(0), dext[:3]
