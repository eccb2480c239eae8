"""Host checks of the entry points of linear attention, the norms and the projections with an epilogue: bad arguments are
refused before anything is launched, and calls with nothing to do return at once.  No GPU needed."""
import ctypes

import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm

OK, EINVAL, EALIGN, EUNSUPPORTED, ENOSPACE, EOVERLAP = 0, -1, -2, -6, -7, -9
F32, BF16 = 0, 1
NONE, SILU, GELU = 0, 1, 2
P, I, LL, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float
MB = 1 << 20
AT = [0x10000000 + i * 16 * MB for i in range(20)]  # never dereferenced on these paths


# ---- linear attention ----


class LinearArgs(ctypes.Structure):
    """sdm_linear_args."""
    _fields_ = ([(n, P) for n in ("q", "k", "v", "g")]
                + [(n, LL) for n in ("q_bs", "q_ts", "k_bs", "k_ts", "v_bs", "v_ts", "g_bs", "g_ts")]
                + [(n, P) for n in ("state", "state_out", "lengths", "slots", "o")]
                + [(n, I) for n in ("dtype", "B", "T", "H", "Hk", "dk", "dv", "n_slots")] + [("scale", F)])


LINEAR = dict(q=AT[0], k=AT[1], v=AT[2], g=AT[3], q_bs=128, q_ts=32, k_bs=128, k_ts=32, v_bs=256, v_ts=64, g_bs=16, g_ts=4,
              state=AT[4], state_out=AT[5], lengths=AT[6], slots=AT[7], o=AT[8], dtype=F32, B=2, T=4, H=4, Hk=2, dk=16, dv=16,
              n_slots=2, scale=0.25)


def linear(ws=0, ws_bytes=0, err=None, **kw):
    f = sdm.lib().sdm_linear_attention
    f.argtypes = [P, P, SZ, P, P]
    return f(ctypes.byref(LinearArgs(**{**LINEAR, **kw})), ws, ws_bytes, err, None)


def test_linear_refusals():
    f = sdm.lib().sdm_linear_attention
    f.argtypes = [P, P, SZ, P, P]
    assert f(None, None, 0, None, None) == EINVAL
    for kw in (dict(B=0), dict(T=-1), dict(H=0), dict(dk=0), dict(dv=0), dict(Hk=0), dict(Hk=3), dict(dtype=2),
               dict(n_slots=0), dict(slots=0, n_slots=1)):
        assert linear(**kw) == EINVAL, kw
    for kw in (dict(dk=257), dict(dv=257), dict(B=1 << 16, T=1 << 16, n_slots=1 << 16), dict(T=0x7FFFFFFF - 64, B=1),
               dict(B=1 << 20, H=1 << 10, Hk=1, T=4, n_slots=1 << 20)):
        assert linear(**kw) == EUNSUPPORTED, kw
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(q=AT[0] + 2), dict(o=AT[8] + 2), dict(state=AT[4] + 2),
               dict(state_out=AT[5] + 1), dict(g=AT[3] + 2), dict(lengths=AT[6] + 1), dict(slots=AT[7] + 2),
               dict(dtype=BF16, v=AT[2] + 1)):
        assert linear(**kw) == EALIGN, kw
    assert linear(T=0, state_out=AT[4]) == OK and linear(T=0, state_out=0, q=0, k=0, v=0, o=0) == OK
    long = dict(B=1, T=4096, n_slots=1)
    need = sdm.linear_attention_workspace_size(torch.float32, 1, 4096, 4, 2, 16, 16)
    assert need > 0 and linear(**long) == EALIGN
    assert linear(ws=AT[9], ws_bytes=need - 1, **long) == ENOSPACE
    assert linear(ws=AT[9] + 8, ws_bytes=need, **long) == EALIGN


def test_linear_workspace_sizes():
    size = sdm.linear_attention_workspace_size
    for ty in (torch.float32, torch.bfloat16):
        assert size(ty, 1, 1, 4, 4, 64, 64) == 0                       # a token
        assert size(ty, 0, 64, 4, 4, 64, 64) == 0 and size(ty, 1, 64, 4, 3, 64, 64) == 0 and size(ty, 1, 64, 4, 4, 257, 8) == 0
        assert size(ty, 64, 4096, 64, 64, 128, 128) == 0               # heads enough
        assert size(ty, 1, 1 << 20, 64, 64, 256, 256) % 16 == 0
    # copies of q, k, v and o in rows of multiples of 8
    assert size(torch.bfloat16, 64, 512, 64, 8, 60, 60) >= 64 * 512 * 2 * (2 * 8 * 64 + 2 * 64 * 64)


def test_linear_refuses_outputs_over_another_tensor():
    names = ("q", "k", "v", "g", "state", "lengths", "slots")
    for T in (1, 4):
        for out in ("o", "state_out"):
            for name in names:
                if (out, name) == ("state_out", "state"):
                    continue
                assert linear(**{out: LINEAR[name]}, T=T) == EOVERLAP, (out, name, T)
                assert linear(**{out: LINEAR[name] - 16}, T=T) == EOVERLAP, (out, name, T)
        assert linear(o=AT[5], T=T) == EOVERLAP
        assert linear(state_out=AT[4] + 16 * 16 * 4 * 4, T=T) == EOVERLAP   # the next sequence's row
    need = sdm.linear_attention_workspace_size(torch.float32, 1, 4096, 4, 2, 16, 16)
    long = dict(B=1, T=4096, n_slots=1)
    for name in (*names, "o", "state_out"):
        assert linear(ws=LINEAR[name], ws_bytes=need, **long) == EOVERLAP, name


# ---- norms ----


class NormArgs(ctypes.Structure):
    """sdm_norm_args."""
    _fields_ = ([(n, P) for n in ("x", "residual", "gate")] + [(n, LL) for n in ("x_rs", "residual_rs", "gate_rs")]
                + [(n, P) for n in ("after", "scale", "weight")] + [(n, I) for n in ("x_dtype", "r_dtype", "w_dtype", "act")]
                + [("M", LL), ("D", I), ("groups", I), ("eps", F)])


class NormGrads(ctypes.Structure):
    """sdm_norm_grads."""
    _fields_ = ([(n, P) for n in ("r", "dy", "dr")] + [(n, LL) for n in ("r_rs", "dy_rs", "dr_rs")]
                + [(n, P) for n in ("dx", "dresidual", "dgate", "dafter", "dscale", "dweight")])


NORM = dict(x=AT[0], residual=AT[1], gate=AT[2], x_rs=64, residual_rs=64, gate_rs=128, after=AT[3], scale=AT[4], weight=AT[5],
            x_dtype=BF16, r_dtype=F32, w_dtype=F32, act=SILU, M=10, D=64, groups=1, eps=1e-6)
GRADS = dict(r=AT[6], dy=AT[7], dr=AT[8], r_rs=64, dy_rs=64, dr_rs=64, dx=AT[9], dresidual=AT[10], dgate=AT[11], dafter=AT[12],
             dscale=AT[13], dweight=AT[14])


def norm(y=AT[15], r=AT[16], **kw):
    f = sdm.lib().sdm_residual_norm
    f.argtypes = [P, P, P, P]
    return f(ctypes.byref(NormArgs(**{**NORM, **kw})), y, r, None)


def norm_grad(ws=AT[17], ws_bytes=None, grads={}, **kw):
    f = sdm.lib().sdm_residual_norm_backward
    f.argtypes = [P, P, P, SZ, P]
    a = {**NORM, **kw}
    need = sdm.residual_norm_backward_workspace_size(a["M"], a["D"], a["groups"]) if ws_bytes is None else ws_bytes
    return f(ctypes.byref(NormArgs(**a)), ctypes.byref(NormGrads(**{**GRADS, **grads})), ws, need, None)


BAD = (dict(M=-1), dict(D=0), dict(groups=0), dict(groups=3), dict(groups=2), dict(x_dtype=2), dict(r_dtype=-1),
       dict(w_dtype=7), dict(act=GELU), dict(eps=-1.0), dict(eps=float("nan")))


def test_norm_refusals():
    for kw in BAD:
        assert norm(**kw) == EINVAL and norm_grad(ws_bytes=1 << 30, **kw) == EINVAL, kw
    for kw in (dict(x_dtype=F32, r_dtype=BF16), dict(D=16400), dict(M=1 << 32)):
        assert norm(**kw) == EUNSUPPORTED and norm_grad(ws_bytes=1 << 30, **kw) == EUNSUPPORTED, kw
    assert norm(y=None) == EINVAL and norm(weight=0) == EINVAL and norm(y=None, r=None, weight=0) == EINVAL
    for kw in (dict(x=0), dict(x=AT[0] + 1), dict(gate=AT[2] + 1), dict(residual=AT[1] + 2), dict(after=AT[3] + 2),
               dict(scale=AT[4] + 1), dict(weight=AT[5] + 2), dict(y=AT[15] + 1), dict(r=AT[16] + 2)):
        assert norm(**kw) == EALIGN, kw
    assert norm(M=0, x=0) == OK
    f = sdm.lib().sdm_residual_norm
    f.argtypes = [P, P, P, P]
    assert f(None, None, None, None) == EINVAL


def test_norm_gradient_refusals():
    for g in (dict(dy=0), dict(r=0)):
        assert norm_grad(grads=g) == EINVAL, g
    assert norm_grad(weight=0) == EINVAL                                     # dweight, and dy, of no weight
    assert norm_grad(weight=0, grads=dict(dweight=0)) == EINVAL
    assert norm_grad(weight=0, grads=dict(dweight=0, dy=0, dr=0)) == EINVAL
    for name in ("after", "scale", "gate"):
        assert norm_grad(**{name: 0}) == EINVAL, name
    assert norm_grad(x=0) == EINVAL
    for g in (dict(dx=AT[9] + 1), dict(dgate=AT[11] + 1), dict(dresidual=AT[10] + 2), dict(dafter=AT[12] + 2),
              dict(dweight=AT[14] + 1), dict(dy=AT[7] + 1), dict(dr=AT[8] + 2), dict(r=AT[6] + 1)):
        assert norm_grad(grads=g) == EALIGN, g
    need = sdm.residual_norm_backward_workspace_size(10, 64, 1)
    assert need > 0 and norm_grad(ws_bytes=need - 1) == ENOSPACE
    assert norm_grad(ws=None) == EALIGN and norm_grad(ws=AT[17] + 8) == EALIGN
    assert sdm.residual_norm_backward_workspace_size(0, 64) == 0
    assert sdm.residual_norm_backward_workspace_size(5, 64, 3) == 0


def test_norm_refuses_outputs_over_another_tensor():
    """y and r may be exactly where rows of their size are; nowhere else."""
    for out in ("y", "r"):
        for name in ("x", "residual", "gate", "after", "scale", "weight"):
            assert norm(**{out: NORM[name] + 32}) == EOVERLAP, (out, name)
    assert norm(y=NORM["gate"]) == EOVERLAP                                  # half of a wider projection
    assert norm(y=NORM["residual"]) == EOVERLAP                              # rows of another size
    assert norm(y=AT[15], r=AT[15] + 16) == EOVERLAP
    outs = ("dx", "dresidual", "dgate", "dafter", "dscale", "dweight")
    ins = dict({n: NORM[n] for n in ("x", "gate", "after", "scale", "weight")}, **{n: GRADS[n] for n in ("r", "dy", "dr")})
    for out in outs:
        for name, at in ins.items():
            assert norm_grad(grads={out: at + 32}) == EOVERLAP, (out, name)
        for other in outs:
            if other != out:
                assert norm_grad(grads={out: GRADS[other] + 16}) == EOVERLAP, (out, other)
        assert norm_grad(ws=GRADS[out]) == EOVERLAP, out
    for name, at in ins.items():
        assert norm_grad(ws=at) == EOVERLAP, name


# ---- projections ----


def project(x=AT[0], w=AT[1], bias=AT[2], residual=AT[3], M=40, D=64, N=128, act=GELU, y=AT[4], ws=AT[5], n=MB, err=None):
    f = sdm.lib().sdm_project
    f.argtypes = [P, P, P, P, LL, I, I, I, P, P, SZ, P, P]
    return f(x, w, bias, residual, M, D, N, act, y, ws, n, err, None)


def project_grad(x=AT[0], w=AT[1], bias=AT[2], dy=AT[3], M=40, D=64, N=128, act=GELU, dx=AT[4], dw=AT[5], dbias=AT[6],
                 ws=AT[7], n=4 * MB):
    f = sdm.lib().sdm_project_backward
    f.argtypes = [P, P, P, P, LL, I, I, I, P, P, P, P, SZ, P, P]
    return f(x, w, bias, dy, M, D, N, act, dx, dw, dbias, ws, n, None, None)


def test_project_refusals():
    for call in (project, project_grad):
        for kw in (dict(M=-1), dict(D=0), dict(N=0), dict(act=-1), dict(act=3)):
            assert call(**kw) == EINVAL, kw
        for kw in (dict(D=60), dict(N=124), dict(M=1 << 31)):
            assert call(**kw) == EUNSUPPORTED, kw
        for kw in (dict(x=None), dict(w=None), dict(x=AT[0] + 8), dict(w=AT[1] + 8), dict(bias=AT[2] + 8)):
            assert call(**kw) == EALIGN, kw
    assert project(y=None) == EALIGN and project(residual=AT[3] + 8) == EALIGN and project(M=0, x=None, y=None) == OK
    assert project_grad(dy=None) == EALIGN and project_grad(dx=AT[4] + 8) == EALIGN and project_grad(dw=None) == EALIGN
    assert project_grad(dbias=AT[6] + 2) == EALIGN and project_grad(ws=None) == EALIGN
    need = sdm.project_workspace_size(40, 4096, 128)
    assert need > 0 and project(D=4096, n=need - 1) == ENOSPACE and project(D=4096, ws=None, n=need) == EALIGN
    assert sdm.project_workspace_size(8, 4096, 128) == 0 and sdm.project_workspace_size(-1, 64, 64) == 0
    need = sdm.project_backward_workspace_size(40, 64, 128, "gelu")
    assert need >= 40 * 128 * 2 and project_grad(n=need - 1) == ENOSPACE
    assert sdm.project_backward_workspace_size(0, 64, 128, "gelu") == 0


def test_project_refuses_outputs_over_another_tensor():
    for M in (4, 40):
        for name, at in (("x", AT[0]), ("w", AT[1]), ("bias", AT[2])):
            assert project(M=M, y=at) == EOVERLAP and project(M=M, y=at - 16) == EOVERLAP, (name, M)
        assert project(M=M, y=AT[3] + 16) == EOVERLAP                        # not exactly the residual
    for name, at in (("x", AT[0]), ("w", AT[1]), ("bias", AT[2]), ("residual", AT[3]), ("y", AT[4])):
        assert project(D=4096, ws=at) == EOVERLAP, name
    outs = dict(dx=AT[4], dw=AT[5], dbias=AT[6], ws=AT[7])
    ins = dict(x=AT[0], w=AT[1], bias=AT[2], dy=AT[3])
    for out in outs:
        for name, at in {**ins, **outs}.items():
            if name != out:
                assert project_grad(**{out: at}) == EOVERLAP, (out, name)
    assert project_grad(M=0, x=None, dy=None, dx=None, dw=AT[1]) == EOVERLAP


def test_python_calls_refuse_host_tensors():
    x, w = torch.zeros(2, 3, 1, 8), torch.zeros(8)
    flat = x.view(6, 8)
    for call in (lambda: sdm.linear_attention(x, x, x), lambda: sdm.linear_attention_step(x[0], x[0], x[0], state=x),
                 lambda: sdm.residual_norm(flat, weight=w), lambda: sdm.gated_norm(flat, w),
                 lambda: sdm.residual_norm_backward(flat, flat, flat, flat, w), lambda: sdm.gated_norm_backward(flat, w, flat),
                 lambda: sdm.project(flat, torch.zeros(8, 8)), lambda: sdm.project_backward(flat, torch.zeros(8, 8), flat)):
        with pytest.raises(TypeError):
            call()
