"""The 64-bit gradient that the GPU tests of the gated projections compare with (layers_ref.py), against central
differences of the 64-bit forward.  No GPU needed.

For a step e the difference of a smooth function is off by e^2 / 6 of its third derivative and by 2^-53 of the
function's size over e: with e = 1e-4 in inputs of size 1 and a loss of some tens of terms of size 1, under 1e-6 of
the gradient's norm times the direction's.  A slope without one of its two terms is off by tenths of it."""
import numpy as np
import pytest

import layers_ref as ref


def _setup(seed):
    rs = np.random.RandomState(seed)
    return rs.standard_normal((12, 24)), rs.standard_normal((2 * 16, 24)) / 24 ** 0.5, rs.standard_normal((12, 16)), rs


def _worst(act, seed):
    """Worst distance of a directional derivative from the differences', in units of the gradient's norm times the
    direction's; over single entries and random directions of x and w."""
    x, w, dh, rs = _setup(seed)
    dx, dw, _, _ = ref.gated_grad(x, w, dh, act)
    loss = lambda a, b: float((ref.gated(a, b, act)[0] * dh).sum())  # noqa: E731
    worst, e = 0.0, 1e-4
    for n in range(16):
        for which, grad in ((0, dx), (1, dw)):
            v = np.zeros_like(grad)
            if n < 8:
                v = rs.standard_normal(grad.shape)
                v /= np.linalg.norm(v)
            else:
                v.flat[rs.randint(v.size)] = 1.0
            step = (e * v, 0.0) if which == 0 else (0.0, e * v)
            diff = (loss(x + step[0], w + step[1]) - loss(x - step[0], w - step[1])) / (2 * e)
            worst = max(worst, abs(diff - float((grad * v).sum())) / np.linalg.norm(grad))
    return worst


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_reference_gradient_is_the_derivative(act):
    for seed in range(4):
        assert _worst(act, seed) < 1e-6


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_wrong_reference_gradient_is_seen(act, monkeypatch):
    good, gate = ref.act_and_slope, ref.gated_grad
    wrong = {
        "slope without its second term": lambda g, a: (good(g, a)[0], good(g, a)[0] / g),
        "slope of one": lambda g, a: (good(g, a)[0], np.ones_like(g)),
        "slope a percent off": lambda g, a: (good(g, a)[0], 1.01 * good(g, a)[1]),
    }
    for name, f in wrong.items():
        monkeypatch.setattr(ref, "act_and_slope", f)
        assert _worst(act, 0) > 1e-4, name
    monkeypatch.setattr(ref, "act_and_slope", good)
    monkeypatch.setattr(ref, "gated_grad", lambda *a: tuple(0.5 * v for v in gate(*a)))
    assert _worst(act, 0) > 1e-2
