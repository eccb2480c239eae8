"""The projections with bias, activation and residual, and their gradient, against the 64-bit definition (mixer_ref.py,
which derives the tolerances; test_mixer_ref.py holds its gradient to differences)."""
import numpy as np
import pytest
import torch

import mixer_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu


def _host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(M, D, N, seed=2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (rn(M, D).bfloat16(), (rn(N, D) * D ** -0.5).bfloat16(), rn(N).bfloat16(), rn(M, N).bfloat16(),
            rn(M, N).bfloat16())


def _check(got, want, bound, label):
    g = _host(got)
    assert g.shape == want.shape
    tol = bound + ref.ROUND["bf16"] * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float(np.nanmax(np.abs(g - want) / tol)):.2f} of the tolerance, first at "
                           f"{tuple(int(i) for i in np.argwhere(bad)[0])}")


SIZES = [
    # M, D, N: few tokens, tiles, tiles with a split reduction
    (1, 8, 8), (1, 64, 136), (3, 72, 40), (8, 2048, 264), (9, 1032, 72), (16, 4096, 24), (16, 520, 2000),
    (17, 128, 136), (33, 1024, 64), (64, 200, 256), (100, 72, 136), (129, 128, 256), (257, 96, 520), (300, 640, 88),
    (20, 4096, 264), (130, 2056, 520), (600, 1000, 1000),
]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("parts", ["", "b", "r", "br"])
@pytest.mark.parametrize("M,D,N", SIZES)
def test_project_against_its_definition(M, D, N, parts, act):
    x, w, bias, residual, _ = _inputs(M, D, N)
    bias, residual = bias if "b" in parts else None, residual if "r" in parts else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sdm.project(x, w, bias, residual, activation=act, dev_err=err)
    want, bound = ref.project(*(_host(t) for t in (x, w, bias, residual)), act)
    assert err.item() == 0
    _check(y, want, bound, "y")
    if residual is not None:
        again = sdm.project(x, w, bias, residual, activation=act, out=residual)   # the stream in place
        assert again is residual and torch.equal(again, y)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("M,D,N", SIZES + [(4096, 64, 64), (2500, 136, 72), (40, 264, 2048)])
def test_project_gradient_against_its_definition(M, D, N, with_bias, act):
    x, w, bias, _, dy = _inputs(M, D, N, seed=7)
    bias = bias if with_bias else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sdm.project_backward(x, w, dy, bias, activation=act, dev_err=err)
    want = ref.project_grad(_host(x), _host(w), _host(bias), _host(dy), act)
    assert err.item() == 0
    for name, t, v, b in zip(("dx", "dw", "dbias"), got, want[:3], want[3:]):
        if name == "dbias" and not with_bias:
            assert t is None
        else:
            _check(t, v, b, name)
    again = sdm.project_backward(x, w, dy, bias, activation=act)
    assert all(u is None or torch.equal(u, v) for u, v in zip(got, again))


# More tiles than the card's 76 pairs of SMs, so that a pair goes on from one to another, with ragged edges.
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("M,D,N", [(5000, 264, 4000), (21003, 136, 1032)])
def test_project_of_more_tiles_than_pairs(M, D, N, act):
    x, w, bias, residual, dy = _inputs(M, D, N, seed=9)
    rows = torch.as_tensor([*range(0, M, M // 60), *range(M - 20, M)], device="cuda")
    y = sdm.project(x, w, bias, residual, activation=act)
    want, bound = ref.project(_host(x[rows]), _host(w), _host(bias), _host(residual[rows]), act)
    _check(y[rows], want, bound, "y")
    dx, dw, db = sdm.project_backward(x, w, dy, bias, activation=act)
    want = ref.project_grad(_host(x[rows]), _host(w), _host(bias), _host(dy[rows]), act)
    _check(dx[rows], want[0], want[3], "dx")
    cols = torch.as_tensor([*range(0, N, N // 30), *range(N - 20, N)], device="cuda")
    want = ref.project_grad(_host(x), _host(w[cols]), _host(bias[cols]), _host(dy[:, cols]), act)
    _check(dw[cols], want[1], want[4], "dw")
    _check(db[cols], want[2], want[5], "dbias")


def test_a_token_does_not_depend_on_the_others():
    """The sums of a tile's tokens run in one order: any split of a batch of more than few tokens gives the same bits
    where the reduction is not split, and padding tokens of NaN reach no other."""
    x, w, bias, residual, _ = _inputs(3000, 128, 4096)
    y = sdm.project(x, w, bias, residual, activation="silu")
    x[5], residual[9] = float("nan"), float("inf")
    z = sdm.project(x, w, bias, residual, activation="silu")
    rest = [i for i in range(3000) if i not in (5, 9)]
    assert torch.equal(y[rest], z[rest]) and torch.isnan(z[5]).all() and torch.isinf(z[9]).all()


def test_project_of_no_tokens_and_extreme_values():
    x, w, bias, residual, dy = _inputs(40, 64, 64)
    x[0] *= 1e4
    for act in ("silu", "gelu"):
        y = sdm.project(x, w, bias, residual, activation=act)
        g = sdm.project_backward(x, w, dy, bias, activation=act)
        assert torch.isfinite(y).all() and all(torch.isfinite(t).all() for t in g)
    for act in ("none", "gelu"):
        assert sdm.project(x[:0], w, bias, residual[:0], activation=act).shape == (0, 64)
        dx, dw, db = sdm.project_backward(x[:0], w, dy[:0], bias, activation=act, dw=torch.full_like(w, 3.0),
                                          dbias=torch.full_like(bias, 3.0))
        assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_project_in_batches_on_other_streams_and_in_graphs():
    x, w, bias, residual, dy = _inputs(60, 1024, 72)
    assert sdm.project_workspace_size(60, 1024, 72) > 0                        # a split reduction
    run = lambda: (sdm.project(x, w, bias, residual, activation="gelu", workspace=wf),  # noqa: E731
                   *sdm.project_backward(x, w, dy, bias, activation="gelu", workspace=wb))
    wf = wb = None
    want = run()
    wf = torch.full((sdm.project_workspace_size(60, 1024, 72),), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((sdm.project_backward_workspace_size(60, 1024, 72, "gelu"),), 255, dtype=torch.uint8, device="cuda")
    three = sdm.project(x.view(3, 20, 1024), w, bias, residual.view(3, 20, 72), activation="gelu")
    assert torch.equal(three.view(60, 72), want[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    few = sdm.project(x[:4], w, bias, residual[:4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
        got_few = sdm.project(x[:4], w, bias, residual[:4])
    for _ in range(2):
        for t in (*got, got_few):
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)) and torch.equal(got_few, few)


def test_project_refuses_what_it_cannot_run():
    x, w, bias, residual, dy = _inputs(40, 64, 64)
    for args, kw in (((x.float(), w), {}), ((x.cpu(), w), {}), ((x, w[:, :-8]), {}), ((x, w, bias[:-1]), {}),
                     ((x, w, bias.float()), {}), ((x, w, None, residual[:-1]), {}), ((x, w), dict(activation="tanh")),
                     ((x[:, ::2], w[:, :32].contiguous()), {})):
        with pytest.raises((TypeError, ValueError)):
            sdm.project(*args, **kw)
    with pytest.raises((TypeError, ValueError)):
        sdm.project_backward(x, w, dy[:-1])
    with pytest.raises(ValueError):
        sdm.project_backward(x, w, dy, dbias=torch.empty_like(bias))
    with pytest.raises(sdm.SDMError):
        sdm.project(x[:, :60].contiguous(), w[:, :60].contiguous())             # D % 8
    with pytest.raises(sdm.SDMError):
        sdm.project(x, w[:60].contiguous())                                    # N % 8
    with pytest.raises(sdm.SDMError):
        sdm.project_backward(x, w, dy, bias, activation="silu", workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for M in (5, 40):
        x, w, bias, residual, dy = _inputs(M, 64, 64)
        kept = x.clone()
        for out in (x, w[:M] if M < 64 else w):
            with pytest.raises(ValueError, match="overlaps"):
                sdm.project(x, w, bias, residual, out=out)
        wide = torch.zeros(M + 1, 64, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ValueError, match="overlaps"):
            sdm.project(x, w, bias, wide[1:], out=wide[:M])
        for outs in (dict(dx=x), dict(dw=w), dict(dx=dy), dict(dbias=bias)):
            with pytest.raises(ValueError, match="overlaps"):
                sdm.project_backward(x, w, dy, bias, **outs)
        assert torch.equal(x, kept)


def test_project_past_32_bit_offsets():
    M, D, N = 270_000, 64, 8192  # 2.2e9 outputs
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((M, D), generator=g, device="cuda").bfloat16()
    w = torch.randn((N, D), generator=g, device="cuda").bfloat16()
    y = sdm.project(x, w, activation="silu")
    assert torch.equal(y[M - 300:], sdm.project(x[M - 300:].contiguous(), w, activation="silu"))
    dx, _, _ = sdm.project_backward(x, w, y, activation="none")
    host = lambda t: t[M - 300:].double().cpu().numpy()  # noqa: E731
    want = ref.project_grad(host(x), w.double().cpu().numpy(), None, host(y), "none")
    _check(dx[M - 300:], want[0], want[3], "dx")


def test_bias_gradient_of_many_tokens():
    """65,537 slices of 256 tokens: sums of ones are exact in fp32, and the total is rounded once."""
    M = 256 * 65536 + 1
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    x[-1] = 1.0
    w = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(M, 8, dtype=torch.bfloat16, device="cuda")
    dx, dw, dbias = sdm.project_backward(x, w, dy, bias=torch.zeros(8, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(dbias.float(), torch.full((8,), 2.0 ** 24, device="cuda"))
    assert torch.equal(dx, dy) and torch.equal(dw, torch.ones_like(dw))


@pytest.mark.parametrize("M,D,N", [(5, 4104, 2008), (2, 2056, 4080), (11, 8192, 48), (16, 6000, 2048)])
def test_few_tokens_of_long_reductions(M, D, N):
    """Blocks of 8 and 16 warps, whose shares of D end anywhere."""
    x, w, bias, residual, _ = _inputs(M, D, N, seed=5)
    want, bound = ref.project(*(_host(t) for t in (x, w, bias, residual)), "gelu")
    _check(sdm.project(x, w, bias, residual, activation="gelu"), want, bound, "y")
