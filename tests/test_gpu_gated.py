"""The gated feed-forward projections and their gradient against the 64-bit definition (layers_ref.py, which derives
the tolerances), and the gradient against differences of the definition."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu


def _host(t):
    return t.detach().double().cpu().numpy()


def _inputs(M, D, F, seed=2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return rn(M, D).bfloat16(), (rn(2 * F, D) * D ** -0.5).bfloat16(), rn(M, F).bfloat16()


def _check(got, want, bound, label):
    g = _host(got)
    assert g.shape == want.shape
    tol = bound + ref.ROUND["bf16"] * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float(np.nanmax(np.abs(g - want) / tol)):.2f} of the tolerance, first at "
                           f"{tuple(int(i) for i in np.argwhere(bad)[0])}")


SIZES = [
    # M, D, F
    (1, 8, 8), (1, 64, 128), (3, 72, 40), (5, 256, 1000), (16, 512, 264), (17, 128, 136), (33, 1024, 64),
    (64, 200, 256), (100, 72, 136), (128, 64, 128), (129, 128, 256), (256, 320, 384), (257, 96, 520),
    (300, 640, 88), (700, 256, 512),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_gated_against_its_definition(M, D, F, act):
    x, w, _ = _inputs(M, D, F)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = sdm.project_gated(x, w, activation=act, dev_err=err)
    want, _, _, bound, _, _ = ref.gated(_host(x), _host(w), act)
    assert err.item() == 0
    _check(h, want, bound, "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", SIZES + [(4096, 64, 64), (2500, 136, 72), (40, 264, 2048)])
def test_gated_gradient_against_its_definition(M, D, F, act):
    x, w, dh = _inputs(M, D, F, seed=7)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = sdm.project_gated_backward(x, w, dh, activation=act, dev_err=err)
    wx, ww, bx, bw = ref.gated_grad(_host(x), _host(w), _host(dh), act)
    assert err.item() == 0
    _check(dx, wx, bx, "dx")
    _check(dw, ww, bw, "dw")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_against_differences(act):
    """Central differences of the 64-bit forward along random directions: for a step e the difference is off by
    e^2 / 6 of the third derivative (under 1e-6 here, of directions of unit size), the gradient by its bf16 parts
    (three roundings of 2^-8, in the mean over many terms far less; their worst case is the tolerance)."""
    x, w, dh = _inputs(24, 64, 96, seed=5)
    dx, dw = sdm.project_gated_backward(x, w, dh, activation=act)
    X, W, H = _host(x), _host(w), _host(dh)
    _, _, bx, bw = ref.gated_grad(X, W, H, act)
    rs = np.random.RandomState(0)
    loss = lambda a, b: float((ref.gated(a, b, act)[0] * H).sum())  # noqa: E731
    for _ in range(4):
        vx, vw = rs.standard_normal(X.shape), rs.standard_normal(W.shape)
        vx, vw = vx / np.linalg.norm(vx), vw / np.linalg.norm(vw)
        e = 1e-4
        gx, gw = _host(dx), _host(dw)
        for diff, got, tol in (
                ((loss(X + e * vx, W) - loss(X - e * vx, W)) / (2 * e), (gx * vx).sum(),
                 (np.abs(vx) * (bx + 2.0 ** -7 * np.abs(gx))).sum()),
                ((loss(X, W + e * vw) - loss(X, W - e * vw)) / (2 * e), (gw * vw).sum(),
                 (np.abs(vw) * (bw + 2.0 ** -7 * np.abs(gw))).sum())):
            assert abs(diff - got) <= tol + 1e-5


def test_gated_of_extreme_gates_and_of_no_tokens():
    x, w, dh = _inputs(40, 64, 64)
    x[0] *= 1e4   # gates of thousands: sigmoid 0 or 1, no overflow
    x[1] = 0.0
    for act in ("silu", "gelu"):
        h = sdm.project_gated(x, w, activation=act)
        dx, dw = sdm.project_gated_backward(x, w, dh, activation=act)
        assert all(torch.isfinite(t).all() for t in (h, dx, dw))
        assert not h[1].any()
    none = x[:0]
    assert sdm.project_gated(none, w).shape == (0, 64)
    dx, dw = sdm.project_gated_backward(none, w, dh[:0], dw=torch.full_like(w, 3.0))
    assert dx.shape == (0, 64) and not dw.any()


def test_gated_takes_batches_outputs_and_other_streams():
    x, w, dh = _inputs(60, 128, 72)
    want, (dx, dw) = sdm.project_gated(x, w), sdm.project_gated_backward(x, w, dh)
    out = torch.full((3, 20, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    assert sdm.project_gated(x.view(3, 20, 128), w, out=out) is out and torch.equal(out.view(60, 72), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.empty(sdm.project_gated_backward_workspace_size(60, 128, 72), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        h2 = sdm.project_gated(x, w)
        dx2, dw2 = sdm.project_gated_backward(x.view(3, 20, 128), w, dh.view(3, 20, 72), workspace=ws)
    side.synchronize()
    assert torch.equal(h2, want) and torch.equal(dx2.view(60, 128), dx) and torch.equal(dw2, dw)


def test_gated_refuses_what_it_cannot_run():
    x, w, dh = _inputs(16, 64, 64)
    with pytest.raises(TypeError):
        sdm.project_gated(x.float(), w)
    with pytest.raises(TypeError):
        sdm.project_gated(x.cpu(), w)
    with pytest.raises(ValueError):
        sdm.project_gated(x, w, activation="none")
    with pytest.raises(ValueError):
        sdm.project_gated(x, w[:-1])
    with pytest.raises(ValueError):
        sdm.project_gated(x[:, ::2], w[:, :32].contiguous())
    with pytest.raises(ValueError):
        sdm.project_gated_backward(x, w, dh[:-1])
    with pytest.raises(sdm.SDMError):
        sdm.project_gated(x[:, :60].contiguous(), w[:, :60].contiguous())   # D % 8
    with pytest.raises(sdm.SDMError):
        sdm.project_gated(x, w[:120].contiguous())                         # F % 8
    with pytest.raises(sdm.SDMError):
        sdm.project_gated_backward(x, w, dh, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_gated_outputs_over_other_tensors():
    """Refused over x, w or one another; dh's memory may take dx, which is written when dh has been read."""
    for M in (5, 300):
        x, w, dh = _inputs(M, 128, 128, seed=9)
        kept = x.clone()
        with pytest.raises(ValueError, match="overlaps"):
            sdm.project_gated(x, w, out=x)
        both = torch.empty(M * 128 + 256 * 128, dtype=torch.bfloat16, device="cuda")
        for outs in (dict(dx=x), dict(dw=w),
                     dict(dx=both[:M * 128].view(M, 128), dw=both[M * 128 - 8:][:256 * 128].view(256, 128))):
            with pytest.raises(ValueError, match="overlaps"):
                sdm.project_gated_backward(x, w, dh, **outs)
        assert torch.equal(x, kept)
        want = sdm.project_gated_backward(x, w, dh)
        dx, dw = sdm.project_gated_backward(x, w, dh, dx=dh)
        assert dx is dh and torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def _check_rows(got, want, label):
    """Row by row in norm: a sum of terms of random sign whose factors dg and du were rounded by up to 2^-8 of themselves,
    evenly, is off by 2^-8 / sqrt(3) of its own size in the mean, and its own rounding adds as much again in squares:
    0.0032 in all, over a row's hundreds of entries.  2^-7 is 2.4 times that; eight wrong entries of a row of 2056 are
    eight times 2^-7."""
    off = np.linalg.norm(_host(got) - want, axis=1) / np.linalg.norm(want, axis=1)
    assert (off < 2.0 ** -7).all(), f"{label}: row {int(off.argmax())} is {float(off.max()):.4f} of its norm off"


def _check_slices(x, w, dh, act, dx, dw, tokens, columns):
    """dx of some tokens and dw of some columns' rows of Wg and Wu (over all tokens) against the 64-bit definition, each
    entry within its bound and each row in norm."""
    F = w.shape[0] // 2
    t = torch.as_tensor(tokens, device="cuda")
    want, _, bound, _ = ref.gated_grad(_host(x[t]), _host(w), _host(dh[t]), act)
    _check(dx[t], want, bound, "dx")
    _check_rows(dx[t], want, "dx")
    f = torch.as_tensor(columns, device="cuda")
    rows = torch.cat([f, f + F])
    _, want, _, bound = ref.gated_grad(_host(x), _host(w[rows]), _host(dh[:, f]), act)
    _check(dw[rows], want, bound, "dw")
    _check_rows(dw[rows], want, "dw")


# The tiles of dx and dw together are more than the card's 76 pairs of SMs, so that a pair goes on from one unit to
# another: both accumulators, ring phases carried over, and a unit of dw after one of dx.
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", [(1000, 1024, 2736), (9000, 264, 4000), (5000, 776, 1304)])
def test_gated_gradient_of_more_tiles_than_pairs(M, D, F, act):
    x, w, dh = _inputs(M, D, F, seed=13)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = sdm.project_gated_backward(x, w, dh, activation=act, dev_err=err)
    assert err.item() == 0
    _check_slices(x, w, dh, act, dx, dw, [*range(0, M, 61), *range(M - 20, M)], [*range(0, F, 53), *range(F - 20, F)])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", [(21003, 1032, 5000), (2000, 2056, 9000), (45000, 520, 4104)])
def test_gated_gradient_of_large_batches(M, D, F, act):
    """608 tiles of dx and dw and more, a launch for each product, with ragged M, D and F."""
    tiles = lambda n: -(-n // 256)  # noqa: E731
    assert tiles(M) * tiles(D) + tiles(2 * F) * tiles(D) >= 608
    x, w, dh = _inputs(M, D, F, seed=15)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = sdm.project_gated_backward(x, w, dh, activation=act, dev_err=err)
    assert err.item() == 0
    _check_slices(x, w, dh, act, dx, dw, [*range(0, M, M // 40), *range(M - 10, M)], [*range(0, F, F // 40), *range(F - 10, F)])
