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

import torch

from . import api as _api
from .api import SDM_BF16, SDM_F32, SDMError

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_CODES = {torch.float32: SDM_F32, torch.bfloat16: SDM_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_c = ctypes
_fns = {}


class _ScanArgs(ctypes.Structure):
    """sdm_ssm_args."""
    _fields_ = ([(n, _c.c_void_p) for n in ("x", "dt", "Bm", "Cm", "z")]
                + [(n, _c.c_longlong) for n in ("x_bs", "x_ts", "dt_bs", "dt_ts", "B_bs", "B_ts", "C_bs", "C_ts",
                                                "z_bs", "z_ts")]
                + [(n, _c.c_void_p) for n in ("A", "D", "dt_bias", "state", "state_out", "lengths", "slots", "y")]
                + [(n, _c.c_int) for n in ("dtype", "B", "T", "Dm", "N", "G", "softplus", "n_slots")])


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(_api.lib(), name)
        p, i, ll, sz = _c.c_void_p, _c.c_int, _c.c_longlong, _c.c_size_t
        f.argtypes, f.restype = {
            "sdm_causal_conv": ([p, ll, ll, i, p, p, i, i, i, i, i, i, p, p, i, p, p, p, p, p], i),
            "sdm_selective_scan": ([_c.POINTER(_ScanArgs), p, sz, p, p], i),
            "sdm_selective_scan_workspace_size": ([i, i, i, i, i], sz),
            "sdm_project_gated": ([p, p, ll, i, i, i, p, p, p], i),
            "sdm_project_gated_backward": ([p, p, p, ll, i, i, i, p, p, p, sz, p, p], i),
            "sdm_project_gated_backward_workspace_size": ([ll, i, i], sz),
        }[name]
        _fns[name] = f
    return f


def _stream(index):
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _refuse(t, name, dtype, shape, index):
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


def _dense(t, name, dtype, shape, index):
    """The address of a contiguous tensor of that type and shape; None for None."""
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != index
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, index)
    return t.data_ptr()


def _rows(t, name, dtype, shape, index):
    """(address, sequence stride, token stride) of a tensor [B, T, ...] whose trailing dimensions are dense; a
    stride of a dimension of one entry does not matter and is given as 0."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(t, name, dtype, shape, index)
    st, n = t.stride(), 1
    for k in range(len(shape) - 1, 1, -1):
        if st[k] != n and shape[k] > 1:
            raise ValueError(f"{name} must be dense in its last {len(shape) - 2} dimension(s)")
        n *= shape[k]
    return t.data_ptr(), (st[0] if shape[0] > 1 else 0), (st[1] if shape[1] > 1 else 0)


def _cuda_index(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return x.get_device()


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation must be one of {', '.join(allowed)}, got {name!r}")
    return ACTIVATIONS[name]


def _state_rows(state, state_out, slots, nb, tail, dtype, index):
    """(address of state, address of state_out, rows, the tensor written): in place where only `state` is given."""
    out = state if state_out is None else state_out
    ref = state if state is not None else out
    if ref is None:
        if slots is not None:
            raise ValueError("slots need a state")
        return None, None, 0, None
    n = ref.shape[0] if isinstance(ref, torch.Tensor) and ref.dim() else 0
    if slots is None and n != nb:
        raise ValueError(f"state must have one row a sequence ({nb}) without slots, got {n}")
    shape = (n, *tail)
    return _dense(state, "state", dtype, shape, index), _dense(out, "state_out", dtype, shape, index), n, out


def causal_conv(x, w, bias=None, state=None, state_out=None, activation="silu", lengths=None, slots=None, out=None,
                dev_err=None):
    """Short causal depthwise convolution over a batch of prompts (sdm_causal_conv):
    y[b,t,d] = act(bias[d] + sum_j w[d,j] u[b,t-K+1+j,d]), u the K-1 carried inputs followed by x.

    x: [B, T, D] fp32 or bf16, rows of any stride (e.g. a slice of a wider projection); w [D, K] and bias [D]
    fp32 or bf16, K from 2 to 8; state, state_out [rows, K-1, D] of x's type, the last K-1 inputs (state None:
    zeros; state_out None: `state` is updated in place, or not kept where there is none).  activation: "silu" or
    "none".  lengths: int32 [B], the tokens of each sequence that exist (y is 0 past them).  slots: int32 [B],
    the row of the state each sequence uses, negative for a padding row.  Returns (y, state written)."""
    index = _cuda_index(x, "x")
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return causal_conv(x, w, bias, state, state_out, activation, lengths, slots, out, dev_err)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    if x.dtype not in _CODES:
        raise TypeError(f"unsupported dtype {x.dtype} (float32 or bfloat16)")
    shape = x.shape
    nb, T, D = shape
    px, bs, ts = _rows(x, "x", x.dtype, shape, index)
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.dtype not in _CODES:
        raise TypeError("w must be a [D, K] float32 or bfloat16 CUDA tensor")
    K = w.shape[1]
    pw = _dense(w, "w", w.dtype, (D, K), index)
    pb = _dense(bias, "bias", w.dtype, (D,), index)
    act = _activation(activation, ("silu", "none"))
    ps, po, rows, written = _state_rows(state, state_out, slots, nb, (K - 1, D), x.dtype, index)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    st = _fn("sdm_causal_conv")(
        px, bs, ts, _CODES[x.dtype], pw, pb, _CODES[w.dtype], nb, T, D, K, act, ps, po, rows,
        _dense(lengths, "lengths", torch.int32, (nb,), index), _dense(slots, "slots", torch.int32, (nb,), index),
        _dense(out, "out", x.dtype, shape, index), _dense(dev_err, "dev_err", torch.int32, (1,), index),
        _stream(index))
    if st != 0:
        raise SDMError("sdm_causal_conv", st)
    return out, written


def causal_conv_step(x, w, bias=None, *, state, state_out=None, activation="silu", slots=None, out=None,
                     dev_err=None):
    """causal_conv for one decode token of every sequence: x [B, D], y [B, D]; the state holds the K-1 inputs before
    it.  Chained steps give what one causal_conv over the same tokens gives, bit for bit."""
    if state is None:
        raise ValueError("a step needs the state")
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [B, D]")
    y, written = causal_conv(x.unsqueeze(1), w, bias, state, state_out, activation, None, slots,
                             None if out is None else out.unsqueeze(1), dev_err)
    return (y.squeeze(1) if out is None else out), written


def selective_scan_workspace_size(B: int, T: int, D: int, N: int, G: int = 1) -> int:
    """Bytes of workspace selective_scan needs for these sizes; 0 where it needs none."""
    return int(_fn("sdm_selective_scan_workspace_size")(B, T, D, N, G))


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, state_out=None, dt_softplus=True,
                   lengths=None, slots=None, out=None, workspace=None, dev_err=None):
    """Selective state space scan over a batch of prompts (sdm_selective_scan):
    h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t h_t + D x_t) silu(z_t),
    delta = softplus(dt + dt_bias) (dt_softplus=False: without the softplus).

    x, dt, z: [B, T, Dm]; B, C: [B, T, N], or [B, T, G, N] where groups of Dm / G channels share them; all of x's
    type (fp32 or bf16), rows of any stride.  A [Dm, N], D [Dm], dt_bias [Dm]: fp32.  N up to 128.  state,
    state_out: fp32 [rows, Dm, N] (state None: zeros; state_out None: `state` is updated in place, or not kept where
    there is none).  lengths, slots: as for causal_conv.  Returns (y of x's type, state written)."""
    index = _cuda_index(x, "x")
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return selective_scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, dt_softplus, lengths, slots, out,
                                  workspace, dev_err)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, Dm]")
    ty = x.dtype
    if ty not in _CODES:
        raise TypeError(f"unsupported dtype {ty} (float32 or bfloat16)")
    shape = x.shape
    nb, T, Dm = shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or not isinstance(B, torch.Tensor) or B.dim() not in (3, 4):
        raise ValueError("A must be [Dm, N] and B and C [B, T, N] or [B, T, G, N]")
    N = A.shape[1]
    G = B.shape[2] if B.dim() == 4 else 1
    bc = (nb, T, G, N) if B.dim() == 4 else (nb, T, N)
    px, x_bs, x_ts = _rows(x, "x", ty, shape, index)
    pd, d_bs, d_ts = _rows(dt, "dt", ty, shape, index)
    pB, b_bs, b_ts = _rows(B, "B", ty, bc, index)
    pC, c_bs, c_ts = _rows(C, "C", ty, bc, index)
    pz, z_bs, z_ts = (None, 0, 0) if z is None else _rows(z, "z", ty, shape, index)
    f32 = torch.float32
    ps, po, rows, written = _state_rows(state, state_out, slots, nb, (Dm, N), f32, index)
    if out is None:
        out = torch.empty(shape, dtype=ty, device=x.device)
    args = _ScanArgs(px, pd, pB, pC, pz, x_bs, x_ts, d_bs, d_ts, b_bs, b_ts, c_bs, c_ts, z_bs, z_ts,
                     _dense(A, "A", f32, (Dm, N), index), _dense(D, "D", f32, (Dm,), index),
                     _dense(dt_bias, "dt_bias", f32, (Dm,), index), ps, po,
                     _dense(lengths, "lengths", torch.int32, (nb,), index),
                     _dense(slots, "slots", torch.int32, (nb,), index), _dense(out, "out", ty, shape, index),
                     _CODES[ty], nb, T, Dm, N, G, 1 if dt_softplus else 0, rows)
    nbytes = 0
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
            _refuse(workspace, "workspace", torch.uint8, None, index)
        nbytes = workspace.numel()
    elif T > 1:
        nbytes = _fn("sdm_selective_scan_workspace_size")(nb, T, Dm, N, G)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    st = _fn("sdm_selective_scan")(_c.byref(args), None if workspace is None else workspace.data_ptr(), nbytes,
                                   _dense(dev_err, "dev_err", torch.int32, (1,), index), _stream(index))
    if st != 0:
        raise SDMError("sdm_selective_scan", st)
    return out, written


def selective_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, state, state_out=None, dt_softplus=True,
                   slots=None, out=None, dev_err=None):
    """selective_scan for one decode token of every sequence: x, dt, z [B, Dm]; B, C [B, N] or [B, G, N]; y [B, Dm]."""
    if state is None:
        raise ValueError("a step needs the state")
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [B, Dm]")
    y, written = selective_scan(x.unsqueeze(1), dt.unsqueeze(1), A, B.unsqueeze(1), C.unsqueeze(1), D,
                                None if z is None else z.unsqueeze(1), dt_bias, state, state_out, dt_softplus, None,
                                slots, None if out is None else out.unsqueeze(1), None, dev_err)
    return (y.squeeze(1) if out is None else out), written


def _gated_args(x, w, index):
    """(tokens, D, F, address of x, address of w) of the gated projections' operands."""
    bf16 = torch.bfloat16
    if x.dim() < 1 or not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] % 2:
        raise ValueError("x must be [..., D] and w [2 * F, D]")
    D = x.shape[-1]
    return (x.numel() // D if D else 0, D, w.shape[0] // 2, _dense(x, "x", bf16, x.shape, index),
            _dense(w, "w", bf16, (w.shape[0], D), index))


def project_gated(x, w, activation="silu", out=None, dev_err=None):
    """Gated feed-forward projections in one kernel: h = act(x Wg^T) * (x Wu^T) (sdm_project_gated).

    x: [..., D] bf16; w: [2*F, D] bf16, one row per output column, Wg's F rows and then Wu's; D and F multiples of
    8.  activation: "silu" or "gelu" (the exact one).  Returns h [..., F] bf16."""
    index = _cuda_index(x, "x")
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return project_gated(x, w, activation, out, dev_err)
    act = _activation(activation, ("silu", "gelu"))
    M, D, F, px, pw = _gated_args(x, w, index)
    shape = (*x.shape[:-1], F)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    st = _fn("sdm_project_gated")(px, pw, M, D, F, act, _dense(out, "out", torch.bfloat16, shape, index),
                                  _dense(dev_err, "dev_err", torch.int32, (1,), index), _stream(index))
    if st != 0:
        raise SDMError("sdm_project_gated", st)
    return out


def project_gated_backward_workspace_size(M: int, D: int, F: int) -> int:
    """Bytes of workspace project_gated_backward needs for M tokens."""
    return int(_fn("sdm_project_gated_backward_workspace_size")(M, D, F))


def project_gated_backward(x, w, dh, activation="silu", dx=None, dw=None, workspace=None, dev_err=None):
    """Gradient of project_gated: (dx [..., D], dw [2*F, D]) for dh [..., F], all bf16
    (sdm_project_gated_backward).  The forward pass keeps nothing but its inputs: the projections are recomputed."""
    index = _cuda_index(x, "x")
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return project_gated_backward(x, w, dh, activation, dx, dw, workspace, dev_err)
    act = _activation(activation, ("silu", "gelu"))
    bf16 = torch.bfloat16
    M, D, F, px, pw = _gated_args(x, w, index)
    ph = _dense(dh, "dh", bf16, (*x.shape[:-1], F), index)
    if dx is None:
        dx = torch.empty(x.shape, dtype=bf16, device=x.device)
    if dw is None:
        dw = torch.empty(w.shape, dtype=bf16, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(16, project_gated_backward_workspace_size(M, D, F)), dtype=torch.uint8,
                                device=x.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        _refuse(workspace, "workspace", torch.uint8, None, index)
    st = _fn("sdm_project_gated_backward")(
        px, pw, ph, M, D, F, act, _dense(dx, "dx", bf16, x.shape, index), _dense(dw, "dw", bf16, w.shape, index),
        workspace.data_ptr(), workspace.numel(), _dense(dev_err, "dev_err", torch.int32, (1,), index),
        _stream(index))
    if st != 0:
        raise SDMError("sdm_project_gated_backward", st)
    return dx, dw
