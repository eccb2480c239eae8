"""The 64-bit gradients that the norms' and projections' kernels are held to, against differences of the 64-bit forward,
and the linear attention's recurrence against its sum over pairs of tokens.  No GPU needed."""
import numpy as np
import pytest

import mixer_ref as ref


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("parts", ["all", "stream", "heads", "gate"])
def test_norm_gradient_against_differences(parts, act):
    rs = np.random.RandomState(3)
    M, D = 3, 12
    groups = 3 if parts == "heads" else 1
    rn = lambda *s: rs.standard_normal(s)  # noqa: E731
    a = dict(x=rn(M, D), residual=rn(M, D) if parts in ("all", "stream") else None,
             weight=rn(D) if parts in ("all", "stream") else None, after=rn(D) if parts in ("all", "heads") else None,
             gate=rn(M, D) if parts != "stream" else None, scale=rn(D) if parts in ("all", "gate") else None)
    gy, gr = rn(M, D), rn(M, D)

    def loss(**kw):
        y, r, _, _ = ref.norm(**{**a, **kw}, groups=groups, eps=1e-3, act=act)
        return (0.0 if y is None else (y * gy).sum()) + (r * gr).sum()

    r = ref.norm(**a, groups=groups, eps=1e-3, act=act)[1]
    got = ref.norm_grad(a["x"], r, gy if a["weight"] is not None else None, gr, a["weight"], a["after"], a["gate"],
                        a["scale"], groups, 1e-3, act)
    for name, v in a.items():
        if v is None:
            continue
        for _ in range(3):
            u = rn(*v.shape)
            diff = (loss(**{name: v + 1e-5 * u}) - loss(**{name: v - 1e-5 * u})) / 2e-5
            want = (got["d" + name] * u).sum()
            assert abs(diff - want) < 1e-6 * (1 + abs(want)), name  # e^2 / 6 of a third derivative of about 1e2


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_project_gradient_against_differences(act):
    rs = np.random.RandomState(5)
    rn = lambda *s: rs.standard_normal(s)  # noqa: E731
    a, gy = dict(x=rn(5, 7), w=rn(6, 7), bias=rn(6)), rn(5, 6)
    dx, dw, db, *_ = ref.project_grad(a["x"], a["w"], a["bias"], gy, act)
    loss = lambda **kw: (ref.project(**{**a, **kw}, residual=None, act=act)[0] * gy).sum()  # noqa: E731
    for name, got in (("x", dx), ("w", dw), ("bias", db)):
        u = rn(*a[name].shape)
        diff = (loss(**{name: a[name] + 1e-5 * u}) - loss(**{name: a[name] - 1e-5 * u})) / 2e-5
        assert abs(diff - (got * u).sum()) < 1e-6 * (1 + abs(diff)), name


def test_linear_recurrence_is_the_sum_over_pairs():
    rs = np.random.RandomState(7)
    B, T, H, Hk, dk, dv = 2, 9, 4, 2, 3, 5
    q, k, v = rs.standard_normal((B, T, Hk, dk)), rs.standard_normal((B, T, Hk, dk)), rs.standard_normal((B, T, H, dv))
    g, S0 = -rs.random_sample((B, T, H)), rs.standard_normal((B, H, dk, dv))
    o, S, _, _ = ref.linear(q, k, v, g, 0.5, S0)
    G = np.cumsum(g, 1)
    for b in range(B):
        for h in range(H):
            for t in range(T):
                want = np.exp(G[b, t, h]) * q[b, t, h // 2] @ S0[b, h]
                for j in range(t + 1):
                    want = want + np.exp(G[b, t, h] - G[b, j, h]) * (q[b, t, h // 2] @ k[b, j, h // 2]) * v[b, j, h]
                assert np.allclose(o[b, t, h], 0.5 * want, rtol=1e-12, atol=1e-12)
