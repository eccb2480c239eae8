"""The layers that stand beside the memory layer in a recurrent stack: the short causal convolution, the selective
state space scan, linear attention, the gated feed-forward projections, and what joins them, norms with gates and
residuals and projections with an epilogue (include/sdm.h, second half).

As in ``api``, every step runs in libsdm.so's CUDA kernels on the current stream, and a tensor that is not on a CUDA
device is refused.  The tensors are checked and the outputs allocated in ``csrc/sdm_binding.cpp``: these calls are on a
decode step's path.

dev_err, where a call takes it, is an int32 [1] tensor that error bits (SDM_DEV_*) are OR-ed into.  After SDM_DEV_TIMEOUT, when
a wait inside a kernel ran out, outputs are unspecified and a state may still be the one from before the call, which nothing
else tells a caller that updates states in place.
"""
from __future__ import annotations

import importlib.util

import torch

from . import api as _api
from . import build as _build

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_module = None


def _binding():
    """The compiled binding (built in-tree on first use if absent or stale)."""
    global _module
    if _module is None:
        _api.lib()
        spec = importlib.util.spec_from_file_location("_layers", _build.build_binding())
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.set_error(_api.SDMError)
        _module = m
    return _module


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation must be one of {', '.join(allowed)}, got {name!r}")
    return ACTIVATIONS[name]


def causal_conv(x, w, bias=None, state=None, state_out=None, activation="silu", lengths=None, slots=None, out=None,
                dev_err=None):
    """Short causal depthwise convolution over a batch of prompts (sdm_causal_conv):
    y[b,t,d] = act(bias[d] + sum_j w[d,j] u[b,t-K+1+j,d]), u the K-1 carried inputs followed by x.

    x: [B, T, D] fp32 or bf16, rows of any stride (e.g. a slice of a wider projection); w [D, K] and bias [D]
    fp32 or bf16, K from 2 to 8; state, state_out [rows, K-1, D] of x's type, the last K-1 inputs (state None:
    zeros; state_out None: `state` is updated in place, or not kept where there is none).  activation: "silu" or
    "none".  lengths: int32 [B], the tokens of each sequence that exist (y is 0 past them).  slots: int32 [B],
    the row of the state each sequence uses, negative for a padding row.  A batch of no sequences has an empty y.
    out: y's memory; it may be x itself up to 8 tokens, and overlaps no other tensor of the call (nor does state_out,
    but for `state` itself): ValueError.  Returns (y, state written)."""
    return (_module or _binding()).conv(x, w, bias, state, state_out, _activation(activation, ("silu", "none")),
                                        lengths, slots, out, dev_err, 2)


def causal_conv_step(x, w, bias=None, *, state, state_out=None, activation="silu", slots=None, out=None,
                     dev_err=None):
    """causal_conv for one decode token of every sequence: x [B, D], y [B, D]; the state holds the K-1 inputs before
    it.  Chained steps give what one causal_conv over the same tokens gives, bit for bit."""
    if state is None:
        raise ValueError("a step needs the state")
    return (_module or _binding()).conv(x, w, bias, state, state_out, _activation(activation, ("silu", "none")),
                                        None, slots, out, dev_err, 1)


def selective_scan_workspace_size(B: int, T: int, D: int, N: int, G: int = 1) -> int:
    """Bytes of workspace selective_scan needs for these sizes; 0 where it needs none."""
    return int(_api.lib().sdm_selective_scan_workspace_size(B, T, D, N, G))


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, state_out=None, dt_softplus=True,
                   lengths=None, slots=None, out=None, workspace=None, dev_err=None):
    """Selective state space scan over a batch of prompts (sdm_selective_scan):
    h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t h_t + D x_t) silu(z_t),
    delta = softplus(dt + dt_bias) (dt_softplus=False: without the softplus).

    x, dt, z: [B, T, Dm]; B, C: [B, T, N], or [B, T, G, N] where groups of Dm / G channels share them; all of x's
    type (fp32 or bf16), rows of any stride.  A [Dm, N], D [Dm], dt_bias [Dm]: fp32.  N up to 128.  state,
    state_out: fp32 [rows, Dm, N] (state None: zeros; state_out None: `state` is updated in place, or not kept where
    there is none).  lengths, slots, an empty batch: as for causal_conv.  out: y's memory; it may be x, dt or z itself,
    and overlaps no other tensor of the call (nor does state_out, but for `state` itself): ValueError.  Returns (y of
    x's type, state written)."""
    return (_module or _binding()).scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, lengths, slots,
                                        out, workspace, dev_err, 2)


def selective_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, state, state_out=None, dt_softplus=True,
                   slots=None, out=None, dev_err=None):
    """selective_scan for one decode token of every sequence: x, dt, z [B, Dm]; B, C [B, N] or [B, G, N]; y [B, Dm]."""
    if state is None:
        raise ValueError("a step needs the state")
    return (_module or _binding()).scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, None, slots,
                                        out, None, dev_err, 1)


def project_gated(x, w, activation="silu", out=None, dev_err=None):
    """Gated feed-forward projections in one kernel: h = act(x Wg^T) * (x Wu^T) (sdm_project_gated).

    x: [..., D] bf16; w: [2*F, D] bf16, one row per output column, Wg's F rows and then Wu's; D and F multiples of
    8.  activation: "silu" or "gelu" (the exact one).  Returns h [..., F] bf16, in `out` where it is given (not over
    x or w: ValueError)."""
    return (_module or _binding()).gated(x, w, _activation(activation, ("silu", "gelu")), out, dev_err)


def project_gated_backward_workspace_size(M: int, D: int, F: int) -> int:
    """Bytes of workspace project_gated_backward needs for M tokens."""
    return int(_api.lib().sdm_project_gated_backward_workspace_size(M, D, F))


def project_gated_backward(x, w, dh, activation="silu", dx=None, dw=None, workspace=None, dev_err=None):
    """Gradient of project_gated: (dx [..., D], dw [2*F, D]) for dh [..., F], all bf16
    (sdm_project_gated_backward).  The forward pass keeps nothing but its inputs: the projections are recomputed.
    dx, dw, workspace: memory for them, which overlaps neither x and w nor one another (ValueError); dx and dw may
    take dh's."""
    return (_module or _binding()).gated_grad(x, w, dh, _activation(activation, ("silu", "gelu")), dx, dw, workspace,
                                              dev_err)


def linear_attention_workspace_size(dtype, B: int, T: int, H: int, Hk: int, dk: int, dv: int) -> int:
    """Bytes of workspace linear_attention needs for q, k, v of torch type `dtype`; 0 where it needs none."""
    code = _api.SDM_BF16 if dtype == torch.bfloat16 else _api.SDM_F32
    return int(_api.lib().sdm_linear_attention_workspace_size(code, B, T, H, Hk, dk, dv))


def linear_attention(q, k, v, decay=None, scale=None, state=None, state_out=None, lengths=None, slots=None, out=None,
                     workspace=None, dev_err=None):
    """Linear attention with a decay for each head over a batch of prompts (sdm_linear_attention):
    S_t = exp(decay_t) S_{t-1} + k_t v_t^T,  o_t = scale q_t S_t.

    q, k: [B, T, Hk, dk]; v: [B, T, H, dv], Hk dividing H (heads h with the same h // (H / Hk) share their queries and
    keys); fp32 or bf16, a token's heads dense, tokens and sequences of any stride.  decay: fp32 logarithms, [B, T, H] of
    any strides between tokens and sequences, [H] (the same for every token) or None; at most 0 where nothing is to
    grow, -inf forgets everything before.  scale: dk ** -0.5 if None.  dk and dv up to 256.  state, state_out: fp32
    [rows, H, dk, dv] (state None: zeros; state_out None: `state` is updated in place, or not kept where there is none).
    lengths, slots, an empty batch: as for causal_conv.  out: o's memory; it overlaps no other tensor of the call (nor does
    state_out, but for `state` itself): ValueError.  Returns (o [B, T, H, dv], state written).

    bf16 prompts with dk up to 128 run in chunks of 128 tokens on the tensor cores, everything else token by token; states
    are fp32 in both.  In chunks an infinity in v makes NaN of its column of the state.  There is no gradient: outputs require
    none, whatever the inputs require (as for the convolution and the scan)."""
    return (_module or _binding()).linear(q, k, v, decay, scale, state, state_out, lengths, slots, out, workspace, dev_err,
                                          2)


def linear_attention_step(q, k, v, decay=None, scale=None, *, state, state_out=None, slots=None, out=None, dev_err=None):
    """linear_attention for one decode token of every sequence: q, k [B, Hk, dk]; v, o [B, H, dv]; decay [B, H], [H] or
    None."""
    if state is None:
        raise ValueError("a step needs the state")
    return (_module or _binding()).linear(q, k, v, decay, scale, state, state_out, None, slots, out, None, dev_err, 1)


def residual_norm(x, residual=None, weight=None, *, after=None, gate=None, scale=None, groups=1, eps=1e-6,
                  activation="silu", out=None, residual_out=None):
    """The norms after and before a block with its gate, residual scale and residual in one pass (sdm_residual_norm):
    a = x / rms(x) * after * act(gate),  r = residual + scale * a,  y = r / rms(r) * weight.

    Every operand but x may be None: its factor, term or norm is left out.  x, gate: [..., D] fp32 or bf16, and residual
    of x's type or fp32: dense rows one stride apart.  after, scale, weight: [D], of one type, fp32 or bf16.  groups: the
    norm of x is over each of `groups` groups of channels (its heads); it needs `weight` None.  activation of the gate:
    "silu" or "none".  A group (a row) has up to 16384 channels.  out, residual_out: memory for y and r, each of
    which may be an input of the same row size (the stream updated in place); otherwise they overlap nothing: ValueError.
    Returns (y of x's type, or None without a weight; r of residual's type, x itself where nothing changes it)."""
    return (_module or _binding()).norm(x, residual, weight, after, gate, scale, out, residual_out, groups, eps,
                                        _activation(activation, ("silu", "none")))


def residual_norm_backward_workspace_size(M: int, D: int, groups: int = 1) -> int:
    """Bytes of workspace residual_norm_backward (and gated_norm_backward) needs for M rows."""
    return int(_api.lib().sdm_residual_norm_backward_workspace_size(M, D, groups))


def residual_norm_backward(x, r, dy, dr=None, weight=None, *, after=None, gate=None, scale=None, residual=True, groups=1,
                           eps=1e-6, activation="silu", workspace=None):
    """Gradient of residual_norm (sdm_residual_norm_backward): (dx, dresidual, dweight, dafter, dgate, dscale), None for
    what the call does not have.

    r: what the forward call returned (None where it was x itself, or without a weight); dy: y's gradient, with a
    weight; dr: the gradient that reaches r from elsewhere, or None.  residual: whether there was one.  Without after, gate and
    scale, dx and dresidual are the same values, and one tensor where their types are the same.  The weights' gradients are
    summed in fp32 in an order that sizes alone decide."""
    return (_module or _binding()).norm_grad(x, r, dy, dr, weight, after, gate, scale, residual, workspace, groups, eps,
                                             _activation(activation, ("silu", "none")))


def gated_norm(x, weight, gate=None, groups=1, eps=1e-6, activation="silu", out=None):
    """x / rms(x) * weight * act(gate), the norm over each of `groups` groups of channels (an attention's heads before its
    last projection): residual_norm's first half.  Returns y of x's type and shape."""
    if weight is None:
        raise ValueError("a norm needs its weight")
    return (_module or _binding()).norm(x, None, None, weight, gate, None, None, out, groups, eps,
                                        _activation(activation, ("silu", "none")))[1]


def gated_norm_backward(x, weight, dy, gate=None, groups=1, eps=1e-6, activation="silu", workspace=None):
    """Gradient of gated_norm: (dx, dweight, dgate), dgate None without a gate."""
    if weight is None:
        raise ValueError("a norm needs its weight")
    g = (_module or _binding()).norm_grad(x, None, None, dy, None, weight, gate, None, False, workspace, groups, eps,
                                          _activation(activation, ("silu", "none")))
    return g[0], g[3], g[4]


def project_workspace_size(M: int, D: int, N: int) -> int:
    """Bytes of workspace project needs for M tokens; 0 where it needs none."""
    return int(_api.lib().sdm_project_workspace_size(M, D, N))


def project(x, w, bias=None, residual=None, activation="none", out=None, workspace=None, dev_err=None):
    """A projection with bias, activation and residual in one kernel: y = residual + act(x w^T + bias) (sdm_project).

    x: [..., D]; w: [N, D]; bias: [N]; residual: [..., N]; all bf16 and dense; D and N multiples of 8.  activation:
    "none", "silu" or "gelu" (the exact one).  out: y's memory; it may be the residual itself, and overlaps nothing else:
    ValueError.  Returns y [..., N] bf16."""
    return (_module or _binding()).dense(x, w, bias, residual, _activation(activation, ("none", "silu", "gelu")), out,
                                         workspace, dev_err)


def project_backward_workspace_size(M: int, D: int, N: int, activation="none") -> int:
    """Bytes of workspace project_backward needs for M tokens."""
    act = _activation(activation, ("none", "silu", "gelu"))
    return int(_api.lib().sdm_project_backward_workspace_size(M, D, N, act))


def project_backward(x, w, dy, bias=None, activation="none", dx=None, dw=None, dbias=None, workspace=None, dev_err=None):
    """Gradient of project for dy [..., N] (sdm_project_backward): (dx [..., D], dw [N, D], dbias [N] or None without a
    bias), all bf16.  The residual's gradient is dy itself.  The forward pass keeps nothing but its inputs: with an activation the
    projection is formed again.  dx, dw, dbias, workspace: memory for them, which overlaps nothing (ValueError)."""
    return (_module or _binding()).dense_grad(x, w, dy, bias, _activation(activation, ("none", "silu", "gelu")), dx, dw,
                                              dbias, workspace, dev_err)
