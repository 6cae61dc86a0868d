"""Differentiable entry points over libkda.

``chunk_kda`` and ``chunk_gdn`` take keyword arguments named as in the chunk_kda
call of the cuLA page ("cuLA(CUDA Linear Attention): NVIDIA Blackwell, Hopper
GPU를 위한 선형 어텐션 고성능 CUDA 커널 라이브러리", section "cuLA 설치 및
사용법"), where the output is then differentiated with ``o.backward(do)``.  The
forward pass is kda_fwd / gdn_fwd and the backward pass kda_bwd / gdn_bwd of the
C ABI; when an input needs a gradient the forward pass is kda_fwd_save /
gdn_fwd_save, which keeps in a workspace what the backward pass would otherwise
recompute, and the backward pass kda_bwd_saved / gdn_bwd_saved reuses it.  That
forward pass is the two-stage one (its records are what the backward pass
needs), so with a gradient requested o differs from kda_fwd's single-launch o
by rounding only.
This module only checks and forwards arguments (no arithmetic of the method
runs outside the library).

``chunk_la`` (linear attention with a decay for each head) and ``gated_norm``
(the norm behind an attention block) are the same over la_fwd / la_bwd and
gated_norm_fwd / gated_norm_bwd; their backward passes need nothing of the
forward call, so they keep the inputs only.

The kernels fix the variant the pages describe as the fast path: q and k are
L2-normalised inside, the KDA gate is formed inside from g, A_log and dt_bias
(clamped at ``lower_bound``), KDA beta arrives as logits and goes through the
sigmoid inside, and the state is [N, H, K, V].  Flags asking for anything else
are rejected.
"""
from __future__ import annotations

from . import _binding as _b


def _torch():
    import torch

    return torch


def _require(flag, want, name, what):
    if bool(flag) != want:
        raise NotImplementedError(f"{name}={flag!r} is not supported: {what}")


class _KDA:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class KDAFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, q, k, v, g, beta, A_log, dt_bias, initial_state, scale,
                            lower_bound, cu_seqlens, output_final_state):
                    ctx.workspace = None
                    if any(ctx.needs_input_grad):
                        # keep what the backward pass would recompute
                        o, final, ctx.workspace = _b.kda_fwd_save(
                            q, k, v, g, beta, A_log, dt_bias, lower_bound, scale, initial_state,
                            output_final_state, cu_seqlens)
                    else:
                        o, final = _b.kda_fwd(q, k, v, g, beta, A_log, dt_bias, lower_bound,
                                              scale, initial_state, output_final_state,
                                              cu_seqlens)
                    ctx.save_for_backward(q, k, v, g, beta, A_log, dt_bias, initial_state,
                                          cu_seqlens)
                    ctx.scale, ctx.lower_bound = scale, lower_bound
                    ctx.dt_shape = dt_bias.shape
                    if final is None:
                        return o
                    return o, final

                @staticmethod
                def backward(ctx, do, dfinal=None):
                    q, k, v, g, beta, A_log, dt_bias, h0, cu = ctx.saved_tensors
                    need = ctx.needs_input_grad
                    # the workspace lives as long as the graph (a second backward
                    # pass under retain_graph reuses it)
                    args = (q, k, v, g, beta, A_log, dt_bias, do.contiguous())
                    kw = dict(lower_bound=ctx.lower_bound, scale=ctx.scale, initial_state=h0,
                              dfinal=None if dfinal is None else dfinal.contiguous(),
                              cu_seqlens=cu, need_dh0=h0 is not None and need[7])
                    if ctx.workspace is not None:
                        r = _b.kda_bwd_saved(*args, ctx.workspace, **kw)
                    else:
                        r = _b.kda_bwd(*args, **kw)
                    return (r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], r["dA_log"],
                            r["ddt_bias"].view(ctx.dt_shape), r["dh0"], None, None, None, None)

            cls.fn = KDAFunction
        return cls.fn


class _GDN:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class GDNFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, q, k, v, g, beta, initial_state, scale, cu_seqlens,
                            output_final_state):
                    ctx.workspace = None
                    if any(ctx.needs_input_grad):
                        o, final, ctx.workspace = _b.gdn_fwd_save(
                            q, k, v, g, beta, scale, initial_state, output_final_state,
                            cu_seqlens)
                    else:
                        o, final = _b.gdn_fwd(q, k, v, g, beta, scale, initial_state,
                                              output_final_state, cu_seqlens)
                    ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
                    ctx.scale = scale
                    if final is None:
                        return o
                    return o, final

                @staticmethod
                def backward(ctx, do, dfinal=None):
                    q, k, v, g, beta, h0, cu = ctx.saved_tensors
                    need = ctx.needs_input_grad
                    args = (q, k, v, g, beta, do.contiguous())
                    kw = dict(scale=ctx.scale, initial_state=h0,
                              dfinal=None if dfinal is None else dfinal.contiguous(),
                              cu_seqlens=cu, need_dh0=h0 is not None and need[5])
                    if ctx.workspace is not None:
                        r = _b.gdn_bwd_saved(*args, ctx.workspace, **kw)
                    else:
                        r = _b.gdn_bwd(*args, **kw)
                    return (r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], r["dh0"], None, None,
                            None)

            cls.fn = GDNFunction
        return cls.fn


def chunk_kda(q, k, v, g, beta, A_log, dt_bias, scale=None, initial_state=None,
              output_final_state=False, lower_bound=-5.0, cu_seqlens=None,
              use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True,
              use_beta_sigmoid_in_kernel=True, safe_gate=True, transpose_state_layout=False):
    """Differentiable chunked KDA.  q, k, g [B,T,H,K] bf16; v [B,T,H,V] bf16; beta
    logits [B,T,H] bf16; A_log [H] fp32; dt_bias [H,K] or [H*K] fp32;
    initial_state [N,H,K,V] fp32 or None; cu_seqlens int32 [N+1] or None (B = 1).
    Returns (o, final_state); final_state is None unless ``output_final_state``.
    Gradients reach q, k, v, g, beta, A_log, dt_bias and initial_state."""
    _require(use_qk_l2norm_in_kernel, True, "use_qk_l2norm_in_kernel",
             "q and k are always L2-normalised in the kernel")
    _require(use_gate_in_kernel, True, "use_gate_in_kernel",
             "the gate is always formed in the kernel from g, A_log and dt_bias")
    _require(use_beta_sigmoid_in_kernel, True, "use_beta_sigmoid_in_kernel",
             "KDA beta is taken as logits and passed through the sigmoid in the kernel")
    _require(safe_gate, True, "safe_gate", "the gate is always clamped at lower_bound")
    _require(transpose_state_layout, False, "transpose_state_layout",
             "states are [N, H, K, V]")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    out = _KDA.get().apply(q, k, v, g, beta, A_log, dt_bias, initial_state, float(scale),
                           float(lower_bound), cu_seqlens, bool(output_final_state))
    return out if output_final_state else (out, None)


def chunk_gdn(q, k, v, g, beta, scale=None, initial_state=None, output_final_state=False,
              cu_seqlens=None, use_qk_l2norm_in_kernel=True):
    """Differentiable chunked gated delta rule (scalar gate per head and token).
    g is the fp32 log decay [B,T,H] (<= 0); beta are probabilities [B,T,H] bf16.
    Other arguments and the result as chunk_kda; gradients reach q, k, v, g, beta
    and initial_state."""
    _require(use_qk_l2norm_in_kernel, True, "use_qk_l2norm_in_kernel",
             "q and k are always L2-normalised in the kernel")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    out = _GDN.get().apply(q, k, v, g, beta, initial_state, float(scale), cu_seqlens,
                           bool(output_final_state))
    return out if output_final_state else (out, None)


class _LA:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class LAFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, q, k, v, log_decay, initial_state, scale, cu_seqlens,
                            output_final_state):
                    o, final = _b.la_fwd(q, k, v, log_decay, scale, initial_state,
                                         output_final_state, cu_seqlens)
                    ctx.save_for_backward(q, k, v, log_decay, initial_state, cu_seqlens)
                    ctx.scale = scale
                    if final is None:
                        return o
                    return o, final

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, do, dfinal=None):
                    q, k, v, log_decay, h0, cu = ctx.saved_tensors
                    r = _b.la_bwd(q, k, v, log_decay, do.contiguous(), ctx.scale, h0,
                                  None if dfinal is None else dfinal.contiguous(), cu,
                                  need_dh0=h0 is not None and ctx.needs_input_grad[4])
                    return r["dq"], r["dk"], r["dv"], None, r["dh0"], None, None, None

            cls.fn = LAFunction
        return cls.fn


class _GatedNorm:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class GatedNormFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, gate, weight, residual, residual_scale, activation, eps):
                    ctx.save_for_backward(x, gate, weight, residual, residual_scale)
                    ctx.activation, ctx.eps = activation, eps
                    return _b.gated_norm_fwd(x, gate, weight, activation, eps, residual,
                                             residual_scale)

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dy):
                    x, gate, weight, residual, residual_scale = ctx.saved_tensors
                    r = _b.gated_norm_bwd(x, gate, weight, dy.contiguous(), ctx.activation,
                                          ctx.eps, residual, residual_scale)
                    return (r["dx"], r["dgate"], r["dweight"], r["dresidual"],
                            r["dresidual_scale"], None, None)

            cls.fn = GatedNormFunction
        return cls.fn


def chunk_la(q, k, v, log_decay, scale=None, initial_state=None, output_final_state=False,
             cu_seqlens=None):
    """Differentiable linear attention with a decay for each head.  q, k [B,T,H,K], v
    [B,T,H,V] bf16, used as given; log_decay [H] fp32 (<= 0); initial_state [N,H,K,V] fp32
    or None; cu_seqlens int32 [N+1] or None (B = 1).  Returns (o, final_state);
    final_state is None unless ``output_final_state``.  Gradients reach q, k, v and
    initial_state; the decays are fixed, so a log_decay that asks for one is refused."""
    torch = _torch()
    if torch.is_grad_enabled() and log_decay.requires_grad:
        raise NotImplementedError("log_decay.requires_grad is not supported: the decays are "
                                  "fixed and get no gradient")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    out = _LA.get().apply(q, k, v, log_decay, initial_state, float(scale), cu_seqlens,
                          bool(output_final_state))
    return out if output_final_state else (out, None)


def gated_norm(x, gate, weight, activation="sigmoid", eps=1e-6, residual=None,
               residual_scale=None):
    """Differentiable gated norm on rows x [..., H, D] (see gated_norm_fwd).  Gradients
    reach x, gate, weight, residual and residual_scale."""
    return _GatedNorm.get().apply(x, gate, weight, residual, residual_scale, activation,
                                  float(eps))


class _GatedScan:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class GatedScanFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, g, input_gate, A_log, dt_bias, initial_state, cu_seqlens,
                            output_final_state, recording):
                    args = (x, g, input_gate, A_log, dt_bias, initial_state, output_final_state,
                            cu_seqlens)
                    states = None
                    if recording and any(ctx.needs_input_grad):
                        # keep what the backward pass needs
                        o, final, states = _b.gated_scan_fwd_save(*args)
                    else:
                        o, final = _b.gated_scan_fwd(*args)
                    ctx.save_for_backward(x, g, input_gate, A_log, dt_bias, states, initial_state,
                                          cu_seqlens)
                    ctx.set_materialize_grads(False)
                    if final is None:
                        return o
                    return o, final

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, do, dfinal=None):
                    x, g, input_gate, A_log, dt_bias, states, h0, cu = ctx.saved_tensors
                    do = torch.zeros_like(x) if do is None else do.contiguous()
                    r = _b.gated_scan_bwd(x, g, input_gate, A_log, dt_bias, do, states,
                                          h0, None if dfinal is None else dfinal.contiguous(), cu,
                                          need_dh0=h0 is not None and ctx.needs_input_grad[5])
                    return (r["dx"], r["dg"], r["dinput_gate"], r["dA_log"], r["ddt_bias"],
                            r["dh0"], None, None, None)

            cls.fn = GatedScanFunction
        return cls.fn


class _ShortConv:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class ShortConvFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, weight, bias, initial_state, activation, cu_seqlens,
                            output_final_state):
                    y, final = _b.short_conv_fwd(x, weight, bias, activation, initial_state,
                                                 output_final_state, cu_seqlens)
                    ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
                    ctx.activation = activation
                    ctx.set_materialize_grads(False)
                    if final is None:
                        return y
                    return y, final

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dy, dfinal=None):
                    x, weight, bias, h0, cu = ctx.saved_tensors
                    dy = torch.zeros_like(x) if dy is None else dy.contiguous()
                    r = _b.short_conv_bwd(x, weight, dy, bias, ctx.activation, h0,
                                          None if dfinal is None else dfinal.contiguous(), cu,
                                          need_dh0=h0 is not None and ctx.needs_input_grad[3])
                    return r["dx"], r["dweight"], r["dbias"], r["dh0"], None, None, None

            cls.fn = ShortConvFunction
        return cls.fn


class _LayerNorm:
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class LayerNormFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, weight, bias, residual, eps):
                    y, total = _b.layer_norm_fwd(x, weight, bias, eps, residual)
                    ctx.save_for_backward(total, weight)
                    ctx.eps = eps
                    ctx.has_bias, ctx.has_residual = bias is not None, residual is not None
                    ctx.set_materialize_grads(False)
                    return (y, total) if residual is not None else y

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dy, dsum=None):
                    total, weight = ctx.saved_tensors
                    dy = torch.zeros_like(total) if dy is None else dy.contiguous()
                    r = _b.layer_norm_bwd(total, weight, dy, ctx.eps,
                                          None if dsum is None else dsum.contiguous(),
                                          need_dbias=ctx.has_bias)
                    return (r["dx"], r["dweight"], r["dbias"],
                            r["dx"] if ctx.has_residual else None, None)

            cls.fn = LayerNormFunction
        return cls.fn


def gated_scan(x, g, input_gate, A_log, dt_bias, initial_state=None, output_final_state=False,
               cu_seqlens=None):
    """Differentiable gated linear recurrence over channels (see gated_scan_fwd).  Returns
    (o, final_state); final_state is None unless ``output_final_state``.  Gradients reach x,
    g, input_gate, A_log, dt_bias and initial_state; where none is asked for, the states
    that they need are not kept."""
    # (always through the function: it refuses what it has no rule for, a forward-mode tangent
    # or a batched tensor, where the plain call would drop it; inside of it gradients are off,
    # so whether they are recorded is asked here)
    out = _GatedScan.get().apply(x, g, input_gate, A_log, dt_bias, initial_state, cu_seqlens,
                                 bool(output_final_state), _torch().is_grad_enabled())
    return out if output_final_state else (out, None)


def short_conv(x, weight, bias=None, activation="silu", initial_state=None,
               output_final_state=False, cu_seqlens=None):
    """Differentiable short causal convolution (see short_conv_fwd).  Returns (y,
    final_state); final_state is None unless ``output_final_state``.  Gradients reach x,
    weight, bias and initial_state."""
    out = _ShortConv.get().apply(x, weight, bias, initial_state, activation, cu_seqlens,
                                 bool(output_final_state))
    return out if output_final_state else (out, None)


def layer_norm(x, weight, bias=None, eps=1e-5, residual=None):
    """Differentiable layer norm on rows x [..., D] (see layer_norm_fwd).  Returns (y, u)
    with u = x + residual, or (y, x) without a residual.  Gradients reach x, weight, bias
    and residual, through y and through u."""
    out = _LayerNorm.get().apply(x, weight, bias, residual, float(eps))
    return out if residual is not None else (out, x)
