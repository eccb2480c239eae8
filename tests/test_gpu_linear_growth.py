"""Linear attention whose decays grow: logarithms above 0, moderate in all, with keys and values that are not 0."""
import numpy as np
import pytest
import torch

import mixer_ref as ref
import sparse_state_linear_sdm_gb300 as sdm
from test_gpu_linear import _case, _check, _host, _live

pytestmark = pytest.mark.gpu

U = ref.U


def _bounds(a, chunked):
    """The 64-bit recurrence with its errors where decays are of any sign.  Sizes m follow it with absolute terms.

    Token by token a factor e^g of its own comes from a product with log2 e (its rounding and the constant's: 1.3 |g| U) and
    an exponential of 4 U; the state takes it and the addition, a rounding each: 6 U + 1.3 |g| U.  Within 16 tokens whose sums
    stay below 30 the factors are within 16 U on the way in and out and at most once a tile on the state: under 2 U a
    token and 48 U.  Segments are joined by the factor of a whole sum G: 2.5 |G| U + 12 U, and |G| is at most the sum of |g|.
    8 U + 4 |g| U a token and 64 U hold all of them.  In chunks a weight is a product of at most four exponentials of sums,
    1.3 |sum| U + 4 U each, or of one factor a token as above, and sums of 128 exact products are within 4 * 128 U of their
    sizes: 640 U once.  There the masked products and the state in front are rounded to bf16 as they are read."""
    q, k, v = (_host(a[n]) for n in ("q", "k", "v"))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    g, scale = np.broadcast_to(_host(a["decay"]), (B, T, H)), dk ** -0.5
    of = np.arange(H) // (H // Hk)
    o, eo = np.zeros((B, T, H, dv)), np.zeros((B, T, H, dv))
    out = _host(a["state"]).copy()
    eout = np.zeros_like(out)
    once = 640 if chunked else 64
    for b in range(B):
        S, m, e = out[b].copy(), np.abs(out[b]), np.zeros((H, dk, dv))
        for t in range(T):
            f = np.exp(g[b, t])[:, None, None]
            step = (8 + 4 * np.abs(g[b, t]))[:, None, None]
            add = k[b, t][of][:, :, None] * v[b, t][:, None, :]
            S = f * S + add
            e = f * (e + step * U * m) + once * U * np.abs(add)
            m = f * m + np.abs(add)
            qt = q[b, t][of]
            o[b, t] = scale * np.einsum("hd,hdv->hv", qt, S)
            size = np.einsum("hd,hdv->hv", np.abs(qt), m)
            eo[b, t] = scale * (np.einsum("hd,hdv->hv", np.abs(qt), e) + (5 * dk + 128) * U * size)
            if chunked:
                eo[b, t] += scale * ref.H * (1 + ref.H) * size
        out[b], eout[b] = S, e + once * U * m
    return o, out, eo, eout


def _profile(name, T):
    """The running sum of the logarithms: to +-s and back within a number of tokens."""
    t = np.arange(1, T + 1)
    if name.startswith("wave"):                     # crosses +-30 within 16 tokens and within a chunk
        height, period = {"wave-fast": (35.0, 40.0), "wave-slow": (38.0, 300.0), "wave-low": (14.0, 23.0)}[name]
        return height * np.sin(2 * np.pi * t / period)
    rise, n = {"tile-5": (5.0, 16), "tile-25": (25.0, 16), "tile-40": (40.0, 16), "chunk-5": (5.0, 128),
               "chunk-40": (40.0, 128), "chunk-70": (70.0, 128)}[name]
    x = t % (2 * n) / n                             # up in n tokens, down in the next n
    return rise * np.where(x <= 1, x, 2 - x)


FORMS = {
    "f32": ("f32", 2, 96, 2, 1, 32, 24, "token", True, None, 0, "dense"),
    "f32-odd": ("f32", 1, 90, 2, 2, 50, 37, "token", True, None, 0, "odd"),
    "f32-cut": ("f32", 1, 500, 2, 2, 64, 64, "token", True, None, 0, "dense"),
    "tokens": ("bf16", 2, 140, 2, 2, 64, 64, "token", True, None, 0, "odd"),
    "tiles": ("bf16", 2, 300, 2, 1, 64, 128, "token", True, None, 0, "wide"),
    "tiles-128": ("bf16", 1, 256, 2, 2, 128, 64, "token", True, None, 0, "wide"),
    "tiles-cut": ("bf16", 1, 1100, 2, 2, 128, 128, "token", True, None, 0, "wide"),
    "copied": ("bf16", 1, 700, 2, 1, 100, 36, "token", True, None, 0, "wide"),
}


@pytest.mark.parametrize("profile", ["tile-5", "tile-25", "tile-40", "chunk-5", "chunk-40", "chunk-70", "wave-fast", "wave-slow",
                                     "wave-low"])
@pytest.mark.parametrize("form", FORMS)
def test_growing_decays_with_keys_and_values(form, profile):
    c = FORMS[form]
    a = _case(c, seed=17)
    B, T, H = a["decay"].shape
    total = np.concatenate([[0.0], _profile(profile, T)])
    g = np.repeat(np.diff(total)[None, :, None], B, 0).repeat(H, 2)
    g[:, :, -1] = -g[:, :, -1]                                # the last head falls first
    g += 0.05 * np.random.RandomState(2).randn(B, T, H)
    a["decay"] = torch.from_numpy(g.astype(np.float32)).cuda()
    want, wstate, eo, es = _bounds(a, chunked=form in ("tiles", "tiles-128", "tiles-cut", "copied"))
    assert np.abs(want).max() < 1e36
    o, st = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))
    _check(o, want, eo, c[0], "o")
    live, _ = _live(a)
    _check(st[live], wstate[live], es[live], "f32", "state")
    # and the next token, from that state
    nxt = {**a, "state": st.clone(), **{n: a[n][:, :1] for n in ("q", "k", "v", "decay")}}
    w1, ws1, e1, es1 = _bounds(nxt, chunked=False)
    o1, st1 = sdm.linear_attention(**nxt)
    _check(o1, w1, e1, c[0], "the next token")
    _check(st1, ws1, es1, "f32", "its state")
