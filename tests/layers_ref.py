"""Plain 64-bit forms of the convolution, the selective scan and the gated projections, token by token from their
definitions, each with a bound on the error that fp32 arithmetic may make on the same inputs.

The bounds follow the operations: U = 2^-24 is a unit of fp32 rounding; exp2 and the quotient of the fast silu are
exact to 4 U and 8 U, so an elementwise function of a value v is within 16 U |f(v)| of the exact one at the rounded
argument.  A bf16 result is then rounded once more, by at most 2^-8 of itself."""
import math

import numpy as np

U = 2.0 ** -24
ROUND = {"f32": 2.0 ** -23, "bf16": 2.0 ** -8}


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def softplus(v):
    return np.logaddexp(0.0, v)


def conv(x, w, bias, state, act, lengths=None, slots=None):
    """(y, new state or None, bound of y's error before its last rounding).  x [B,T,D]; state [rows,K-1,D]."""
    B, T, D = x.shape
    K = w.shape[1]
    y, mag = np.zeros((B, T, D)), np.zeros((B, T, D))
    out = None if state is None else state.copy()
    for b in range(B):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        s = b if slots is None else int(slots[b])
        if s < 0:
            continue
        old = np.zeros((K - 1, D)) if state is None else state[s]
        u = np.concatenate([old, x[b, :n]])
        for t in range(n):
            terms = u[t:t + K] * w.T
            y[b, t] = bias + terms.sum(0)
            mag[b, t] = np.abs(bias) + np.abs(terms).sum(0)
        if out is not None:
            out[s] = u[n:]
    if act == "silu":
        v = y
        y = v * sigmoid(v)
        # |silu'| <= 1.1; K + 1 roundings of the sum, then the function's own
        return y, out, 1.1 * (K + 1) * U * mag + 16 * U * np.abs(y) + 8 * U * np.abs(v) * np.abs(y)
    return y, out, (K + 1) * U * mag


def scan(x, dt, A, Bm, Cm, D, z, dt_bias, state, dt_softplus, lengths=None, slots=None):
    """(y, new state, bound of y's error, bound of the state's error).  Bm, Cm [B,T,G,N]; state [rows,Dm,N]."""
    B, T, Dm = x.shape
    G, N = Bm.shape[2], Bm.shape[3]
    y, ey = np.zeros((B, T, Dm)), np.zeros((B, T, Dm))
    out = np.array(state, copy=True)
    eout = np.zeros_like(out)
    for b in range(B):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        s = b if slots is None else int(slots[b])
        if s < 0:
            continue
        h, m, e = out[s].copy(), np.abs(out[s]), np.zeros((Dm, N))
        for t in range(n):
            v = dt[b, t] + (0.0 if dt_bias is None else dt_bias)
            dl = softplus(v) if dt_softplus else v
            # the argument's rounding moves softplus by at most |v| U, its series and functions by 16 U dl
            edl = 2 * U * np.abs(v) + 16 * U * np.abs(dl)
            a = np.exp(dl[:, None] * A)
            Bt = np.repeat(Bm[b, t], Dm // G, axis=0)
            Ct = np.repeat(Cm[b, t], Dm // G, axis=0)
            # relative error of the decay: of its argument, of exp2, and two roundings
            ra = np.abs(A) * edl[:, None] + 3 * U * np.abs(dl[:, None] * A) + 6 * U
            add = np.abs(dl * x[b, t])[:, None] * np.abs(Bt)
            eadd = np.abs(x[b, t] * edl)[:, None] * np.abs(Bt) + 3 * U * add
            e = a * (e + ra * (m + e)) + eadd + 2 * U * (a * m + add)
            h = a * h + (dl * x[b, t])[:, None] * Bt
            m = a * m + add
            o = (h * Ct).sum(1)
            eo = (np.abs(Ct) * e).sum(1) + (N + 2) * U * (np.abs(Ct) * m).sum(1)
            if D is not None:
                o = o + D * x[b, t]
                eo = eo + 2 * U * (np.abs(o) + np.abs(D * x[b, t]))
            if z is not None:
                g = z[b, t] * sigmoid(z[b, t])
                eo = eo * np.abs(g) + (18 + 8 * np.abs(z[b, t])) * U * np.abs(o * g)
                o = o * g
            y[b, t], ey[b, t] = o, eo
        out[s], eout[s] = h, e
    return y, out, ey, eout


def act_and_slope(g, act):
    if act == "silu":
        p = sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    p = 0.5 * np.vectorize(math.erfc)(-g / math.sqrt(2.0))
    return g * p, p + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def gated(x, w, act):
    """(h, g, u, bound of h's error before its rounding, bounds of g's and u's).  D exact products, summed in fp32 in
    any order: within 4 D U of the sum of their sizes."""
    F, D = w.shape[0] // 2, x.shape[1]
    g, u = x @ w[:F].T, x @ w[F:].T
    eg, eu = 4 * D * U * (np.abs(x) @ np.abs(w[:F]).T), 4 * D * U * (np.abs(x) @ np.abs(w[F:]).T)
    a, slope = act_and_slope(g, act)
    ea = (np.abs(slope) + eg) * eg + (16 + 8 * np.abs(g)) * U * np.abs(a)  # |act''| <= 1
    return a * u, g, u, (np.abs(u) + eu) * ea + np.abs(a) * eu + 2 * U * np.abs(a * u), eg, eu


def gated_grad(x, w, dh, act):
    """(dx, dw, bounds of their errors before the last rounding): dg and du are rounded to bf16 on the way."""
    F = w.shape[0] // 2
    _, g, u, _, eg, eu = gated(x, w, act)
    a, s = act_and_slope(g, act)
    ea = (np.abs(s) + eg) * eg + (16 + 8 * np.abs(g)) * U * np.abs(a)
    es = eg + (32 + 16 * np.abs(g)) * U * (1 + np.abs(g))
    d = np.concatenate([dh * u * s, dh * a], axis=1)
    e = np.concatenate([np.abs(dh) * ((np.abs(u) + eu) * es + np.abs(s) * eu), np.abs(dh) * ea], axis=1)
    e = e + (2.0 ** -8 + 4 * U) * (np.abs(d) + e)
    n = 4 * U * (np.abs(d) + e)
    dx, dw = d @ w, d.T @ x
    return dx, dw, (e + 2 * F * n) @ np.abs(w), (e + x.shape[0] * n).T @ np.abs(x)
