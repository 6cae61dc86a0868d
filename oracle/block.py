"""fp64 reference of what stands around an attention block: the gated linear
recurrence over channels, the short causal convolution and the layer norm, each
with its gradients (PyTorch on the CPU; test infrastructure only).

The forward passes are written from the definitions, token by token, and are
differentiable; the gradients are autograd's.  Next to the values stand bounds
on what fp32 arithmetic may lose, by the same recurrences over absolute values.
"""
from __future__ import annotations

import torch

from .linear import spans

# Relative error of one step's factor or term in fp32 (an exponential, a logarithm, a
# square root and a handful of products, each an ulp or two): a step of the recurrence
# may lose this much of its absolute terms.  A decay a = exp(-L) has the error of L on top:
# an fp32 L is off by its own rounding and by those of exp(A_log), of log(1 + e^z), of
# their product and of L / ln 2, at most 4 L 2^-24 together, and a by as much of itself:
# L / 4 times STEP.
STEP = 2.0 ** -20
TINY = 2.0 ** -126  # the smallest normal number of fp32


def _d(t):
    return None if t is None else t.detach().double().cpu()


def gates(x, g, i, A_log, dt_bias):
    """(L, a, m, s) of the recurrence."""
    z = g + dt_bias
    # log(1 + e^z) without overflow; its derivative is the sigmoid
    L = torch.exp(A_log) * torch.logaddexp(z, torch.zeros_like(z))
    # sigmoid(i) = e^-log(1 + e^-i), whose derivative is s sigmoid(-i): s (1 - s) would lose an
    # open gate's slope (at i = 30 it is 9.4e-14, and 64 bits hold s to 1.1e-16)
    s = torch.exp(-torch.logaddexp(-i, torch.zeros_like(i)))
    return L, torch.exp(-L), torch.sqrt(-torch.expm1(-2 * L)), s


def scan(x, g, i, A_log, dt_bias, h0=None, cu=None):
    """(o, final) in fp64, differentiable; rows outside every sequence are zeros."""
    B, T, C = x.shape
    _, a, m, s = gates(x, g, i, A_log, dt_bias)
    u = m * s * x
    sp = spans(B, T, cu)
    rows = [[torch.zeros(C, dtype=torch.float64)] * T for _ in range(B)]
    final = []
    for n, (b, t0, t1) in enumerate(sp):
        h = torch.zeros(C, dtype=torch.float64) if h0 is None else h0[n]
        for t in range(t0, t1):
            h = a[b, t] * h + u[b, t]
            rows[b][t] = h
        final.append(h)
    o = torch.stack([torch.stack(r) if T else torch.zeros(0, C, dtype=torch.float64) for r in rows])
    return o, torch.stack(final)


def scan_all(x, g, i, A_log, dt_bias, h0=None, cu=None, do=None, dfinal=None):
    """Values and bounds: {name: (value, bound)} for o, final and, with ``do``, the
    gradients."""
    x, g, i, A_log, dt_bias, h0, do, dfinal = map(_d, (x, g, i, A_log, dt_bias, h0, do, dfinal))
    B, T, C = x.shape
    sp = spans(B, T, cu)
    N = len(sp)
    if cu is not None:  # rows outside every sequence count for nothing, NaN or not
        keep = torch.zeros(T, dtype=torch.bool)
        for _, t0, t1 in sp:
            keep[t0:t1] = True
        x, g, i = (torch.where(keep[:, None], t, torch.zeros_like(t)) for t in (x, g, i))
        do = None if do is None else torch.where(keep[:, None], do, torch.zeros_like(do))
    names = ["x", "g", "i", "A_log", "dt_bias"] + (["h0"] if h0 is not None else [])
    leaves = dict(x=x, g=g, i=i, A_log=A_log, dt_bias=dt_bias, h0=h0)
    for n in names:
        leaves[n].requires_grad_(do is not None)
    o, final = scan(cu=cu, **leaves)
    L, a, m, s = (t.detach() for t in gates(x, g, i, A_log, dt_bias))
    x, g, i, h0 = (None if t is None else t.detach() for t in (x, g, i, h0))
    # absolute states before each token, and what they may be off by
    z = lambda *sh: torch.zeros(*sh, dtype=torch.float64)  # noqa: E731
    habs, herr, pabs, perr = z(B, T, C), z(B, T, C), z(B, T, C), z(B, T, C)
    fabs, ferr = z(N, C), z(N, C)
    for n, (b, t0, t1) in enumerate(sp):
        mag = z(C) if h0 is None else h0[n].abs()
        err = z(C)
        for t in range(t0, t1):
            pabs[b, t], perr[b, t] = mag, err
            kept = a[b, t] * mag
            mag = kept + (m[b, t] * s[b, t] * x[b, t]).abs()
            err = a[b, t] * err + STEP * (mag + L[b, t] / 4 * kept)
            habs[b, t], herr[b, t] = mag, err
        fabs[n], ferr[n] = mag, err
    out = dict(o=(o.detach(), herr), final=(final.detach(), ferr))
    if do is None:
        return out
    df = z(N, C) if dfinal is None else dfinal
    grads = torch.autograd.grad((o * do).sum() + (final * df).sum(), [leaves[n] for n in names],
                                allow_unused=True)
    grads = {n: z(*leaves[n].shape) if t is None else t for n, t in zip(names, grads)}
    eabs, eerr = z(B, T, C), z(B, T, C)
    dh_err = z(N, C)
    for n, (b, t0, t1) in enumerate(sp):
        mag, err = df[n].abs(), z(C)
        for t in range(t1 - 1, t0 - 1, -1):
            mag = mag + do[b, t].abs()
            err = err + STEP * mag
            eabs[b, t], eerr[b, t] = mag, err
            mag, err = a[b, t] * mag, a[b, t] * (err + STEP * (1 + L[b, t] / 4) * mag)
        dh_err[n] = err
    inv = torch.where(m > 0, 1 / m, torch.zeros_like(m))
    few = 4 * STEP  # the factors that a gradient is multiplied by at the end
    side = a * s * x.abs() * inv + pabs
    p_abs = a * eabs * side
    # A decay below fp32's normal numbers counts as zero there: with a off by TINY, p = a e
    # (a s x / m - h) is off by TINY e (a s x / m + h) (and the second a by as much of s x / m,
    # again times a, which is then below TINY itself).  Times exp(A_log) sigmoid(z), or L,
    # of a hundred it is above the floor that the tests allow by themselves.
    p_err = a * (eerr * side + eabs * perr) + few * (1 + L / 4) * p_abs + TINY * eabs * side
    slope = torch.exp(A_log.detach()) * torch.sigmoid(g + dt_bias.detach())
    out.update(x=(grads["x"], (eerr + few * eabs) * m * s),
               i=(grads["i"], (eerr + few * eabs) * m * x.abs() * s * torch.sigmoid(-i)),
               g=(grads["g"], (p_err + few * p_abs) * slope),
               A_log=(grads["A_log"], ((p_err + few * p_abs) * L).sum((0, 1))),
               dt_bias=(grads["dt_bias"], ((p_err + few * p_abs) * slope).sum((0, 1))))
    out["h0"] = (grads["h0"] if h0 is not None else _scan_dh0(a, do, df, sp), dh_err)
    return out


def _scan_dh0(a, do, df, sp):
    r = df.clone()
    for n, (b, t0, t1) in enumerate(sp):
        for t in range(t1 - 1, t0 - 1, -1):
            r[n] = a[b, t] * (r[n] + do[b, t])
    return r


def conv(x, weight, bias=None, activation="silu", h0=None, cu=None):
    """(y, final, z) in fp64, differentiable; rows outside every sequence are zeros."""
    B, T, C = x.shape
    W = weight.shape[1]
    y = [[torch.zeros(T, C, dtype=torch.float64)] for _ in range(B)]
    z_all = torch.zeros(B, T, C, dtype=torch.float64)
    final = []
    for n, (b, t0, t1) in enumerate(spans(B, T, cu)):
        front = torch.zeros(W - 1, C, dtype=torch.float64) if h0 is None else h0[n]
        ext = torch.cat([front, x[b, t0:t1]])
        z = sum(weight[:, j] * ext[j:j + t1 - t0] for j in range(W))
        if bias is not None:
            z = z + bias
        v = z * torch.sigmoid(z) if activation == "silu" else z
        y[b].append(torch.nn.functional.pad(v, (0, 0, t0, T - t1)))
        z_all[b, t0:t1] = z.detach()
        final.append(ext[t1 - t0:])
    return torch.stack([sum(r) for r in y]), torch.stack(final), z_all


def conv_all(x, weight, bias=None, activation="silu", h0=None, cu=None, dy=None, dfinal=None):
    """{name: (value, bound)} for y, final and, with ``dy``, the gradients."""
    x, weight, bias, h0, dy, dfinal = map(_d, (x, weight, bias, h0, dy, dfinal))
    B, T, C = x.shape
    if cu is not None:
        keep = torch.zeros(T, dtype=torch.bool)
        for _, t0, t1 in spans(B, T, cu):
            keep[t0:t1] = True
        x = torch.where(keep[:, None], x, torch.zeros_like(x))
        dy = None if dy is None else torch.where(keep[:, None], dy, torch.zeros_like(dy))
    leaves = dict(x=x, weight=weight, bias=bias, h0=h0)
    names = [n for n, t in leaves.items() if t is not None]
    for n in names:
        leaves[n].requires_grad_(dy is not None)
    y, final, z = conv(activation=activation, cu=cu, **leaves)
    plain = {n: None if t is None else t.detach() for n, t in leaves.items()}
    size = {n: None if t is None else t.abs() for n, t in plain.items()}
    zabs = conv(activation="none", cu=cu, **size)[2]
    z_err = 8 * 2.0 ** -24 * zabs
    s = torch.sigmoid(z)
    silu = activation == "silu"
    y_err = 1.1 * z_err + STEP * (z * s).abs() if silu else z_err
    out = dict(y=(y.detach(), y_err), final=(final.detach(), torch.zeros_like(final.detach())))
    if dy is None:
        return out
    df = torch.zeros_like(final) if dfinal is None else dfinal
    grads = dict(zip(names, torch.autograd.grad((y * dy).sum() + (final * df).sum(), [leaves[n] for n in names])))
    # |silu''| <= 1/2
    slope = s * (1 + z.abs() * (1 - s)) if silu else torch.ones_like(z)
    dzabs = dy.abs() * slope
    dz_err = dy.abs() * (0.5 * z_err if silu else 0.0) + STEP * dzabs
    # sums of products by the convolution's own gradient, over absolute values and errors

    def spread(dz):
        lv = {n: None if t is None else t.clone().requires_grad_() for n, t in size.items()}
        yy, ff, _ = conv(activation="none", cu=cu, **lv)
        ns = [n for n in lv if lv[n] is not None]
        return dict(zip(ns, torch.autograd.grad((yy * dz).sum() + (ff * df.abs()).sum(), [lv[n] for n in ns],
                                                allow_unused=True)))

    err, mag = spread(dz_err), spread(dzabs)
    for n in names:
        out["d" + n] = (grads[n], err[n] + 4 * STEP * mag[n])
    return out


def layer_norm(u, weight, bias=None, eps=1e-5):
    mean = u.mean(-1, keepdim=True)
    d = u - mean
    y = d / torch.sqrt((d * d).mean(-1, keepdim=True) + eps) * weight
    return y if bias is None else y + bias


def layer_norm_all(u, weight, bias=None, eps=1e-5, dy=None, dsum=None):
    """{name: (value, bound)} for y and, with ``dy``, the gradients (u: what is
    normalised)."""
    u, weight, bias, dy, dsum = map(_d, (u, weight, bias, dy, dsum))
    leaves = [t for t in (u, weight, bias) if t is not None]
    for t in leaves:
        t.requires_grad_(dy is not None)
    y = layer_norm(u, weight, bias, eps)
    v, w = u.detach(), weight.detach()
    d = v - v.mean(-1, keepdim=True)
    std = torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    fine = 2.0 ** -17
    # a difference from the mean is off by an ulp or two of the larger of the two
    n_abs = d.abs() / std
    n_err = 2.0 ** -21 * (v.abs() + v.mean(-1, keepdim=True).abs()) / std + fine * n_abs
    out = dict(y=(y.detach(), n_err * w.abs() + 2.0 ** -22 * (0 if bias is None else bias.detach().abs())))
    if dy is None:
        return out
    total = (y * dy).sum()
    if dsum is not None:
        total = total + (u * dsum).sum()
    grads = torch.autograd.grad(total, leaves)
    t = (dy * w).abs()
    mean = lambda q: q.mean(-1, keepdim=True)  # noqa: E731
    mag = t + mean(t) + n_abs * mean(t * n_abs)
    err = fine * mag + n_err * mean(t * n_abs) + n_abs * mean(t * n_err)
    rows = tuple(range(u.dim() - 1))
    out["dx"] = (grads[0], err / std + 2.0 ** -22 * (0 if dsum is None else dsum.abs()))
    out["dweight"] = (grads[1], (dy.abs() * (n_err + fine * n_abs)).sum(rows))
    if bias is not None:
        out["dbias"] = (grads[2], fine * dy.abs().sum(rows))
    return out
