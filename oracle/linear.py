"""fp64 reference of linear attention with a decay for each head, its gradients,
and the gated norm with its gradients (NumPy; test infrastructure only).

The attention is the token recurrence S_t = a S_{t-1} + k_t v_t^T,
o_t = scale S_t^T q_t, and the gradients its reverse-mode derivative, token by
token; the norm's gradients are the chain rule on each row.
"""
from __future__ import annotations

import numpy as np


def _a64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def spans(B, T, cu=None):
    """(batch row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = [int(x) for x in cu]
    return [(0, c[i], c[i + 1]) for i in range(len(c) - 1)]


def la_fwd(q, k, v, log_decay, scale, h0=None, cu=None):
    q, k, v, ld, h0 = map(_a64, (q, k, v, log_decay, h0))
    B, T, H, K = q.shape
    V = v.shape[3]
    a = np.exp(ld)[:, None, None]
    sp = spans(B, T, cu)
    o = np.zeros((B, T, H, V))
    fin = np.zeros((len(sp), H, K, V))
    for n, (b, t0, t1) in enumerate(sp):
        S = np.zeros((H, K, V)) if h0 is None else h0[n].copy()
        for t in range(t0, t1):
            S = a * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = scale * np.einsum("hkv,hk->hv", S, q[b, t])
        fin[n] = S
    return o, fin


def la_bwd(q, k, v, log_decay, scale, do, h0=None, dfin=None, cu=None):
    q, k, v, ld, h0, do, dfin = map(_a64, (q, k, v, log_decay, h0, do, dfin))
    B, T, H, K = q.shape
    V = v.shape[3]
    a = np.exp(ld)[:, None, None]
    sp = spans(B, T, cu)
    r = dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape),
             dh0=np.zeros((len(sp), H, K, V)))
    for n, (b, t0, t1) in enumerate(sp):
        S = np.zeros((H, K, V)) if h0 is None else h0[n].copy()
        for t in range(t0, t1):
            S = a * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            r["dq"][b, t] = scale * np.einsum("hkv,hv->hk", S, do[b, t])
        E = np.zeros((H, K, V)) if dfin is None else dfin[n].copy()
        for t in range(t1 - 1, t0 - 1, -1):
            E = E + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            r["dv"][b, t] = np.einsum("hkv,hk->hv", E, k[b, t])
            r["dk"][b, t] = np.einsum("hkv,hv->hk", E, v[b, t])
            E = a * E
        r["dh0"][n] = E
    return r


def _act(z, activation):
    s = 1.0 / (1.0 + np.exp(-np.clip(z, -700, 700)))
    return (s, s * (1 - s)) if activation == "sigmoid" else (z * s, s + z * s * (1 - s))


def gated_norm(x, gate, weight, activation, eps, residual=None, residual_scale=None, dy=None):
    """y, or with ``dy`` a dict of y and the gradients."""
    x, gate, weight, residual, residual_scale, dy = map(
        _a64, (x, gate, weight, residual, residual_scale, dy))
    u = x if residual is None else x + residual_scale[:, None] * residual
    D = u.shape[-1]
    root = np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    act, slope = (1.0, 0.0) if gate is None else _act(gate, activation)
    y = u / root * weight * act
    if dy is None:
        return y
    t = dy * weight * act
    dx = t / root - u * (t * u).sum(-1, keepdims=True) / (D * root ** 3)
    rows = tuple(range(u.ndim - 1))
    r = dict(y=y, dx=dx, dweight=(dy * u / root * act).sum(rows))
    if gate is not None:
        r["dgate"] = dy * u / root * weight * slope
    if residual is not None:
        r["dresidual"] = dx * residual_scale[:, None]
        r["dresidual_scale"] = (dx * residual).sum(rows[:-1] + (u.ndim - 1,))
    return r
