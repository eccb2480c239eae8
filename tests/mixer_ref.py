"""Plain 64-bit forms of linear attention, the norms with gate and residual, the projections with an epilogue and their
gradients, each with a bound on the error that the arithmetic named here may make on the same inputs.

U = 2^-24 is a unit of fp32 rounding, H = 2^-8 half a step of bf16 relative to the value (layers_ref.py has the same)."""
import numpy as np

from layers_ref import ROUND, U, act_and_slope, sigmoid  # noqa: F401

H = 2.0 ** -8


# ---- linear attention ----


def linear(q, k, v, g, scale, state, lengths=None, slots=None, chunked=False):
    """(o, new state, bound of o's error before its rounding, bound of the state's).  q, k [B,T,Hk,dk]; v [B,T,H,dv];
    g [B,T,H] logarithms of the decays; state [rows,H,dk,dv].

    Token by token a contribution that has been in the state for n tokens has taken at most one rounding a token and, for every
    16 tokens, factors that are each within 16 U of themselves: under 2 U a token and 48 U besides (two factors on the way in,
    one on the way out).  In chunks (`chunked`) a sum over 128 tokens of exact products is within 4 * 128 U of the sum of their
    sizes whatever its order, the weights within 32 U, and v's three parts leave 2^-24; the masked products and the state in
    front of a chunk are rounded to bf16 as they are read, each by H of itself, and both are at most |q| times the sum of
    the sizes."""
    B, T, Hk, dk = q.shape
    nh, dv = v.shape[2], v.shape[3]
    o, eo = np.zeros((B, T, nh, dv)), np.zeros((B, T, nh, dv))
    out = np.array(state, copy=True)
    eout = np.zeros_like(out)
    of = np.arange(nh) // (nh // Hk)
    step, once = (4 + 2, 4 * 128 + 64) if chunked else (2, 48)
    for b in range(B):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        s = b if slots is None else int(slots[b])
        if s < 0:
            continue
        S, m, e = out[s].copy(), np.abs(out[s]), np.zeros((nh, dk, dv))
        for t in range(n):
            a = np.exp(g[b, t])[:, None, None]
            kt, vt, qt = k[b, t][of], v[b, t], q[b, t][of]
            add = kt[:, :, None] * vt[:, None, :]
            S = np.where(S == 0, 0.0, a * np.where(S == 0, 1.0, S)) + add
            e = a * (e + step * U * m) + once * U * np.abs(add)
            m = a * m + np.abs(add)
            aq = np.abs(qt)
            o[b, t] = scale * np.einsum("hd,hdv->hv", qt, S)
            size = np.einsum("hd,hdv->hv", aq, m)
            eo[b, t] = abs(scale) * (np.einsum("hd,hdv->hv", aq, e) + (dk + 64 + (4 * dk if chunked else 0)) * U * size)
            if chunked:
                eo[b, t] += abs(scale) * H * (1 + H) * size
        out[s], eout[s] = S, e + once * U * m
    return o, out, eo, eout


# ---- norms ----


def _rms(v, groups, eps):
    n = v.shape[-1] // groups
    return np.repeat(np.sqrt((v.reshape(*v.shape[:-1], groups, n) ** 2).mean(-1) + eps), n, axis=-1)


def norm(x, residual, weight, after, gate, scale, groups, eps, act):
    """(y or None, r, bounds of their errors before their roundings).  A sum of squares runs through at most 32 terms in a
    thread and a tree of 10 levels: 48 U, 24 U of the root, and with the root's own and three products 32 U of x / rms *
    after; silu is within 16 U + 8 U |z|; the scale, the addition and a last norm follow."""
    a, ea = x, np.zeros_like(x)
    if after is not None:
        a = x / _rms(x, groups, eps) * after
        ea = 32 * U * np.abs(a)
    if gate is not None:
        s = gate * sigmoid(gate) if act == "silu" else gate
        ea = np.abs(s) * ea + (20 + 8 * np.abs(gate)) * U * np.abs(a * s)
        a = a * s
    if scale is not None:
        a, ea = a * scale, np.abs(scale) * ea + U * np.abs(a * scale)
    r, er = a, ea
    if residual is not None:
        r = residual + a
        er = ea + U * (np.abs(residual) + np.abs(a))
    if weight is None:
        return None, r, None, er
    rms = _rms(r, 1, eps)
    y = r / rms * weight
    # r's errors move y in place and through the mean
    ey = np.abs(weight) / rms * er + np.abs(y) * (np.abs(r) * er).mean(-1, keepdims=True) / rms ** 2 + 40 * U * np.abs(y)
    return y, r, ey, er


def norm_grad(x, r, dy, dr, weight, after, gate, scale, groups, eps, act, size=False):
    """dx, dresidual, dweight, dafter, dgate, dscale as a dict; with `size` their terms' sizes added up instead of the terms.
    A result is within 256 U of that: its factors are some ten, each within 24 U; the sums over rows add a unit a row."""
    A = np.abs if size else (lambda v: v)
    minus = 1.0 if size else -1.0
    out = {}
    d = A(dr) if dr is not None else 0.0
    if weight is not None:
        i = 1.0 / _rms(r, 1, eps)
        u = A(dy) * A(weight)
        out["dweight"] = (A(dy) * A(r) * i).sum(0)
        d = d + i * (u + minus * A(r) * i ** 2 * (u * A(r)).mean(-1, keepdims=True))
    out["dresidual"] = d
    j = 1.0 / _rms(x, groups, eps) if after is not None else 1.0
    n = A(x) * j * (A(after) if after is not None else 1.0)
    s, ds = 1.0, 0.0
    if gate is not None:
        p = sigmoid(gate)
        s = A(gate * p) if act == "silu" else A(gate)
        ds = (p + A(gate) * p * (1 - p) if size else p * (1 + gate * (1 - p))) if act == "silu" else 1.0
    if scale is not None:
        out["dscale"] = (d * n * s).sum(0)
        d = d * A(scale)
    if gate is not None:
        out["dgate"] = d * n * ds
        d = d * s
    if after is not None:
        out["dafter"] = (d * A(x) * j).sum(0)
        u = d * A(after)
        g = x.shape[-1] // groups
        mean = np.repeat((u * A(x)).reshape(*x.shape[:-1], groups, g).mean(-1), g, axis=-1)
        d = j * (u + minus * A(x) * j ** 2 * mean)
    out["dx"] = d
    return out


# ---- projections ----


def project(x, w, bias, residual, act):
    """(y, bound before its rounding).  D exact products summed in fp32 in any order: within 4 D U of the sum of their
    sizes."""
    z = x @ w.T + (0.0 if bias is None else bias)
    ez = 4 * x.shape[1] * U * (np.abs(x) @ np.abs(w).T) + U * np.abs(z)
    if act == "none":
        y, ey = z, ez
    else:
        y, slope = act_and_slope(z, act)
        ey = (np.abs(slope) + ez) * ez + (16 + 8 * np.abs(z)) * U * np.abs(y)
    if residual is not None:
        ey = ey + U * (np.abs(y) + np.abs(residual))
        y = y + residual
    return y, ey


def project_grad(x, w, bias, dy, act):
    """(dx, dw, dbias, bounds before their roundings): with an activation dz is rounded to bf16 on the way."""
    z = x @ w.T + (0.0 if bias is None else bias)
    d, e = dy, np.zeros_like(dy)
    if act != "none":
        ez = 4 * x.shape[1] * U * (np.abs(x) @ np.abs(w).T) + U * np.abs(z)
        _, s = act_and_slope(z, act)
        d = dy * s
        e = np.abs(dy) * (ez + (32 + 16 * np.abs(z)) * U * (1 + np.abs(z)))  # |act''| <= 1
        e = e + H * (np.abs(d) + e)
    n = 4 * U * (np.abs(d) + e)
    M, N = dy.shape
    return (d @ w, d.T @ x, d.sum(0), (e + N * n) @ np.abs(w), (e + M * n).T @ np.abs(x), (e + M * n).sum(0))
