"""Python binding of the layers that stand beside the memory layer in a recurrent stack: the short
causal convolution, the selective state space scan and the gated feed-forward projections
(include/sdm.h, second half).

As in ``api``: argument checks and marshalling only, every step runs in libsdm.so's CUDA kernels
on the current stream, and a tensor that is not on a CUDA device is refused.  The calls are on a
decode step's path, so the checks read plain attributes and the device is switched only where the
tensors are not on the current one.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import api as _api
from .api import SDM_BF16, SDM_F32, SDMError

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_CODES = {torch.float32: SDM_F32, torch.bfloat16: SDM_BF16}
_I32, _FP32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_c = ctypes
_fns = {}

# sdm_ssm_args: x, dt, B, C, z; their strides; A, D, dt_bias, state, state_out, lengths, slots, y; dtype, B, T, Dm,
# N, G, softplus, n_slots
_scan_args = struct.Struct("@5P10q8P8i").pack
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(_api.lib(), name)
        p, i, ll, sz = _c.c_void_p, _c.c_int, _c.c_longlong, _c.c_size_t
        f.argtypes, f.restype = {
            "sdm_causal_conv": ([p, ll, ll, i, p, p, i, i, i, i, i, i, p, p, i, p, p, p, p, p], i),
            "sdm_selective_scan": ([_c.c_char_p, p, sz, p, p], i),
            "sdm_selective_scan_workspace_size": ([i, i, i, i, i], sz),
            "sdm_project_gated": ([p, p, ll, i, i, i, p, p, p], i),
            "sdm_project_gated_backward": ([p, p, p, ll, i, i, i, p, p, p, sz, p, p], i),
            "sdm_project_gated_backward_workspace_size": ([ll, i, i], sz),
        }[name]
        _fns[name] = f
    return f


def _refuse(t, name, dtype, shape, index):
    """Raises what is wrong with t."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}: every tensor of one call must be on the "
                         "same device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _tensor(t, name):
    """t's device index; every entry point starts from its first tensor's."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _dense(t, name, dtype, shape, index):
    """The address of a contiguous tensor of that type and shape; 0 for None."""
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _rows(t, name, dtype, shape, index, lead):
    """(address, sequence stride, token stride) of a tensor [B, T, ...] (lead 2) or [B, ...] (lead 1) whose trailing
    dimensions are dense; a stride over one entry does not matter and is given as 0."""
    try:
        ok = t.dtype is dtype and t.shape == shape and t.get_device() == index
    except AttributeError:
        ok = False
    if not ok:
        _refuse(t, name, dtype, shape, index)
    st = t.stride()
    if len(shape) > lead + 1 or st[lead] != 1:
        n = 1
        for k in range(len(shape) - 1, lead - 1, -1):
            if st[k] != n and shape[k] > 1:
                raise ValueError(f"{name} must be dense in its last {len(shape) - lead} dimension(s)")
            n *= shape[k]
    return (t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if lead == 2 and shape[1] > 1 else 0)


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation must be one of {', '.join(allowed)}, got {name!r}")
    return ACTIVATIONS[name]


def _state_rows(state, state_out, slots, nb, tail, dtype, index):
    """(address of state, address of state_out, rows, the tensor written): in place where only `state` is given."""
    out = state if state_out is None else state_out
    ref = out if state is None else state
    if ref is None:
        if slots is not None:
            raise ValueError("slots need a state")
        return 0, 0, 0, None
    n = ref.shape[0] if isinstance(ref, torch.Tensor) and ref.dim() else 0
    if slots is None and n != nb:
        raise ValueError(f"state must have one row a sequence ({nb}) without slots, got {n}")
    shape = (n, *tail)
    ps = _dense(state, "state", dtype, shape, index)
    return ps, (ps if out is state else _dense(out, "state_out", dtype, shape, index)), n, out


def _conv(x, w, bias, state, state_out, activation, lengths, slots, out, dev_err, lead):
    """causal_conv on [B, T, D] (lead 2) or [B, D] (lead 1)."""
    index = _tensor(x, "x")
    if index != _device():
        with torch.cuda.device(index):
            return _conv(x, w, bias, state, state_out, activation, lengths, slots, out, dev_err, lead)
    shape, ty = x.shape, x.dtype
    if len(shape) != lead + 1:
        raise ValueError("x must be [B, T, D]" if lead == 2 else "x must be [B, D]")
    if ty not in _CODES:
        raise TypeError(f"unsupported dtype {ty} (float32 or bfloat16)")
    nb, D = shape[0], shape[-1]
    T = shape[1] if lead == 2 else 1
    px, bs, ts = _rows(x, "x", ty, shape, index, lead)
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.dtype not in _CODES:
        raise TypeError("w must be a [D, K] float32 or bfloat16 CUDA tensor")
    wt, K = w.dtype, w.shape[1]
    pw = _dense(w, "w", wt, (D, K), index)
    pb = _dense(bias, "bias", wt, (D,), index)
    act = _activation(activation, ("silu", "none"))
    ps, po, rows, written = _state_rows(state, state_out, slots, nb, (K - 1, D), ty, index)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        py = out.data_ptr()
    else:
        py = _dense(out, "out", ty, shape, index)
    st = _fn("sdm_causal_conv")(px, bs, ts, _CODES[ty], pw, pb, _CODES[wt], nb, T, D, K, act, ps, po, rows,
                                _dense(lengths, "lengths", _I32, (nb,), index),
                                _dense(slots, "slots", _I32, (nb,), index), py,
                                _dense(dev_err, "dev_err", _I32, (1,), index), _raw_stream(index))
    if st != 0:
        raise SDMError("sdm_causal_conv", st)
    return out, written


def causal_conv(x, w, bias=None, state=None, state_out=None, activation="silu", lengths=None, slots=None, out=None,
                dev_err=None):
    """Short causal depthwise convolution over a batch of prompts (sdm_causal_conv):
    y[b,t,d] = act(bias[d] + sum_j w[d,j] u[b,t-K+1+j,d]), u the K-1 carried inputs followed by x.

    x: [B, T, D] fp32 or bf16, rows of any stride (e.g. a slice of a wider projection); w [D, K] and bias [D]
    fp32 or bf16, K from 2 to 8; state, state_out [rows, K-1, D] of x's type, the last K-1 inputs (state None:
    zeros; state_out None: `state` is updated in place, or not kept where there is none).  activation: "silu" or
    "none".  lengths: int32 [B], the tokens of each sequence that exist (y is 0 past them).  slots: int32 [B],
    the row of the state each sequence uses, negative for a padding row.  Returns (y, state written)."""
    return _conv(x, w, bias, state, state_out, activation, lengths, slots, out, dev_err, 2)


def causal_conv_step(x, w, bias=None, *, state, state_out=None, activation="silu", slots=None, out=None,
                     dev_err=None):
    """causal_conv for one decode token of every sequence: x [B, D], y [B, D]; the state holds the K-1 inputs before
    it.  Chained steps give what one causal_conv over the same tokens gives, bit for bit."""
    if state is None:
        raise ValueError("a step needs the state")
    return _conv(x, w, bias, state, state_out, activation, None, slots, out, dev_err, 1)


def selective_scan_workspace_size(B: int, T: int, D: int, N: int, G: int = 1) -> int:
    """Bytes of workspace selective_scan needs for these sizes; 0 where it needs none."""
    return int(_fn("sdm_selective_scan_workspace_size")(B, T, D, N, G))


def _scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, lengths, slots, out, workspace, dev_err, lead):
    """selective_scan on [B, T, Dm] (lead 2) or [B, Dm] (lead 1)."""
    index = _tensor(x, "x")
    if index != _device():
        with torch.cuda.device(index):
            return _scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, lengths, slots, out, workspace,
                         dev_err, lead)
    shape, ty = x.shape, x.dtype
    if len(shape) != lead + 1:
        raise ValueError("x must be [B, T, Dm]" if lead == 2 else "x must be [B, Dm]")
    if ty not in _CODES:
        raise TypeError(f"unsupported dtype {ty} (float32 or bfloat16)")
    nb, Dm = shape[0], shape[-1]
    T = shape[1] if lead == 2 else 1
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or not isinstance(B, torch.Tensor):
        raise TypeError("A must be a [Dm, N] and B a [..., N] or [..., G, N] CUDA tensor")
    N = A.shape[1]
    bc = B.shape
    G = bc[lead] if len(bc) == lead + 2 else 1
    if tuple(bc) != (*shape[:-1], G, N) and tuple(bc) != (*shape[:-1], N):
        raise ValueError(f"B must have shape {(*shape[:-1], N)} or {(*shape[:-1], 'G', N)}, got {tuple(bc)}")
    px, x_bs, x_ts = _rows(x, "x", ty, shape, index, lead)
    pd, d_bs, d_ts = _rows(dt, "dt", ty, shape, index, lead)
    pB, b_bs, b_ts = _rows(B, "B", ty, bc, index, lead)
    pC, c_bs, c_ts = _rows(C, "C", ty, bc, index, lead)
    pz, z_bs, z_ts = (0, 0, 0) if z is None else _rows(z, "z", ty, shape, index, lead)
    ps, po, rows, written = _state_rows(state, state_out, slots, nb, (Dm, N), _FP32, index)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        py = out.data_ptr()
    else:
        py = _dense(out, "out", ty, shape, index)
    args = _scan_args(px, pd, pB, pC, pz, x_bs, x_ts, d_bs, d_ts, b_bs, b_ts, c_bs, c_ts, z_bs, z_ts,
                      _dense(A, "A", _FP32, (Dm, N), index), _dense(D, "D", _FP32, (Dm,), index),
                      _dense(dt_bias, "dt_bias", _FP32, (Dm,), index), ps, po,
                      _dense(lengths, "lengths", _I32, (nb,), index), _dense(slots, "slots", _I32, (nb,), index), py,
                      _CODES[ty], nb, T, Dm, N, G, 1 if dt_softplus else 0, rows)
    pw = nbytes = 0
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
            _refuse(workspace, "workspace", torch.uint8, None, index)
        nbytes = workspace.numel()
    elif T > 1:
        nbytes = _fn("sdm_selective_scan_workspace_size")(nb, T, Dm, N, G)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    if nbytes:
        pw = workspace.data_ptr()
    st = _fn("sdm_selective_scan")(args, pw, nbytes, _dense(dev_err, "dev_err", _I32, (1,), index), _raw_stream(index))
    if st != 0:
        raise SDMError("sdm_selective_scan", st)
    return out, written


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, state_out=None, dt_softplus=True,
                   lengths=None, slots=None, out=None, workspace=None, dev_err=None):
    """Selective state space scan over a batch of prompts (sdm_selective_scan):
    h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t h_t + D x_t) silu(z_t),
    delta = softplus(dt + dt_bias) (dt_softplus=False: without the softplus).

    x, dt, z: [B, T, Dm]; B, C: [B, T, N], or [B, T, G, N] where groups of Dm / G channels share them; all of x's
    type (fp32 or bf16), rows of any stride.  A [Dm, N], D [Dm], dt_bias [Dm]: fp32.  N up to 128.  state,
    state_out: fp32 [rows, Dm, N] (state None: zeros; state_out None: `state` is updated in place, or not kept where
    there is none).  lengths, slots: as for causal_conv.  Returns (y of x's type, state written)."""
    return _scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, lengths, slots, out, workspace, dev_err,
                 2)


def selective_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, state, state_out=None, dt_softplus=True,
                   slots=None, out=None, dev_err=None):
    """selective_scan for one decode token of every sequence: x, dt, z [B, Dm]; B, C [B, N] or [B, G, N]; y [B, Dm]."""
    if state is None:
        raise ValueError("a step needs the state")
    return _scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, None, slots, out, None, dev_err, 1)


def _gated_operands(x, w, index):
    """(tokens, D, F, address of x, address of w) of the gated projections' operands."""
    xs = x.shape
    if not xs or not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] % 2:
        raise ValueError("x must be [..., D] and w [2 * F, D]")
    D, F2 = xs[-1], w.shape[0]
    return (x.numel() // D if D else 0, D, F2 // 2, _dense(x, "x", _BF16, xs, index),
            _dense(w, "w", _BF16, (F2, D), index))


def project_gated(x, w, activation="silu", out=None, dev_err=None):
    """Gated feed-forward projections in one kernel: h = act(x Wg^T) * (x Wu^T) (sdm_project_gated).

    x: [..., D] bf16; w: [2*F, D] bf16, one row per output column, Wg's F rows and then Wu's; D and F multiples of
    8.  activation: "silu" or "gelu" (the exact one).  Returns h [..., F] bf16."""
    index = _tensor(x, "x")
    if index != _device():
        with torch.cuda.device(index):
            return project_gated(x, w, activation, out, dev_err)
    act = _activation(activation, ("silu", "gelu"))
    M, D, F, px, pw = _gated_operands(x, w, index)
    shape = (*x.shape[:-1], F)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        ph = out.data_ptr()
    else:
        ph = _dense(out, "out", _BF16, shape, index)
    st = _fn("sdm_project_gated")(px, pw, M, D, F, act, ph, _dense(dev_err, "dev_err", _I32, (1,), index),
                                  _raw_stream(index))
    if st != 0:
        raise SDMError("sdm_project_gated", st)
    return out


def project_gated_backward_workspace_size(M: int, D: int, F: int) -> int:
    """Bytes of workspace project_gated_backward needs for M tokens."""
    return int(_fn("sdm_project_gated_backward_workspace_size")(M, D, F))


def project_gated_backward(x, w, dh, activation="silu", dx=None, dw=None, workspace=None, dev_err=None):
    """Gradient of project_gated: (dx [..., D], dw [2*F, D]) for dh [..., F], all bf16
    (sdm_project_gated_backward).  The forward pass keeps nothing but its inputs: the projections are recomputed."""
    index = _tensor(x, "x")
    if index != _device():
        with torch.cuda.device(index):
            return project_gated_backward(x, w, dh, activation, dx, dw, workspace, dev_err)
    act = _activation(activation, ("silu", "gelu"))
    M, D, F, px, pw = _gated_operands(x, w, index)
    ph = _dense(dh, "dh", _BF16, (*x.shape[:-1], F), index)
    if dx is None:
        dx = torch.empty(x.shape, dtype=_BF16, device=x.device)
    if dw is None:
        dw = torch.empty(w.shape, dtype=_BF16, device=w.device)
    if workspace is None:
        workspace = torch.empty(max(16, project_gated_backward_workspace_size(M, D, F)), dtype=torch.uint8,
                                device=x.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        _refuse(workspace, "workspace", torch.uint8, None, index)
    st = _fn("sdm_project_gated_backward")(
        px, pw, ph, M, D, F, act, _dense(dx, "dx", _BF16, x.shape, index), _dense(dw, "dw", _BF16, w.shape, index),
        workspace.data_ptr(), workspace.numel(), _dense(dev_err, "dev_err", _I32, (1,), index), _raw_stream(index))
    if st != 0:
        raise SDMError("sdm_project_gated_backward", st)
    return dx, dw
