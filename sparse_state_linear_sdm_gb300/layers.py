"""The layers that stand beside the memory layer in a recurrent stack: the short causal convolution, the selective
state space scan and the gated feed-forward projections (include/sdm.h, second half).

As in ``api``, every step runs in libsdm.so's CUDA kernels on the current stream, and a tensor that is not on a CUDA
device is refused.  The tensors are checked and the outputs allocated in ``csrc/sdm_binding.cpp``: these calls are on a
decode step's path.
"""
from __future__ import annotations

import importlib.util

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
